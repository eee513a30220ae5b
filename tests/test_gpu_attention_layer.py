"""The quantized linears, the KV cache and the attention over it in one layer (GPU).

However a text enters, the cache holds the same codes, so its attention outputs
differ by their roundings only: to the output type (half a step each, 2 u |y|) and
of the softmax weights to FP16 (2^-11 mean|v| each), u = 2^-8 for BF16.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DIM, HIDDEN = 128, 512


@pytest.fixture(scope="module")
def mod():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from bit_gemm_w4_amd import attention_layer
    return attention_layer


def _rows(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, HIDDEN, generator=g).to("cuda:0", torch.bfloat16)


def _layer(mod, fmt, **kw):
    return mod.AttentionLayer(HIDDEN, 4, 2, DIM, 1, 512, mod.FORMATS[fmt], page_size=16, **kw)


def _near(a, b, layer):
    from bit_gemm_w4_amd import ops
    _, v = ops.kv_cache_read(layer.cache, layer._ints(layer._slots(0, 0, layer.lens[0]), torch.int64), torch.float32)
    lim = 2.0 ** -7 * torch.maximum(a.abs(), b.abs()).float() + 2.0 ** -9 * v.abs().max()
    assert ((a.float() - b.float()).abs() <= lim).all()


# 1-row projections run in another kernel than many-row ones, so rows are projected once
# and both layers take the same projections.
def _same_projections(layer, x):
    whole = layer._project(x)
    at = 0

    def project(part):
        nonlocal at
        out = tuple(t[at:at + part.shape[0]] for t in whole)
        at += part.shape[0]
        return out
    layer._project = project


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4)])
def test_a_text_in_chunks_or_token_by_token(mod, fmt, window, sinks):
    x = _rows(150, 1)
    outs, caches = [], []
    for counts in ([150], [100, 30] + [1] * 20):
        layer = _layer(mod, fmt, window=window, sinks=sinks)
        _same_projections(layer, x)
        y, at = [], 0
        for n in counts:
            part, _, _ = layer._attend(x[at:at + n], [n])
            layer.lens = [layer.lens[0] + n]
            y.append(part)
            at += n
        outs.append(torch.cat(y))
        caches.append((layer.cache.k.clone(), layer.cache.v.clone(), layer.cache.k_scales.clone(), layer.cache.v_scales.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*caches))
    _near(outs[0], outs[1], layer)


@pytest.mark.parametrize("fmt", ["int8", "fp8", "int4"])
def test_a_checked_tree_is_its_branches(mod, fmt):
    """Each drafted token's output is that of its branch fed as a text, and the accepted branch stays."""
    x, drafts = _rows(90, 2), _rows(6, 3)
    parents = [-1, 0, 0, 2, -1, 3]
    layer = _layer(mod, fmt)
    layer.extend(x, [90])
    k, v, _ = [t.clone() for t in (layer.cache.k, layer.cache.v, layer.cache.k_scales)]
    layer._project = (lambda p: lambda part: p)(layer._project(drafts))
    y = layer._attend(drafts, [6], layer._ints(mod.tree_bits(parents), torch.int64))[0]
    for token in range(6):
        branch = [token]
        while parents[branch[0]] >= 0:
            branch.insert(0, parents[branch[0]])
        other = _layer(mod, fmt)
        other.extend(x, [90])
        rows = torch.tensor(branch).cuda()
        other._project = (lambda p: lambda part: tuple(t[rows] for t in p))(other._project(drafts))
        z, _, _ = other._attend(drafts[rows], [len(branch)])
        other.lens = [90 + len(branch)]
        _near(y[token], z[-1], other)
    layer.check(drafts, [parents])
    layer.accept([[0, 2, 3, 5]])
    assert layer.lens == [94]
    after = _layer(mod, fmt)
    after.extend(x, [90])
    after._project = (lambda p: lambda part: tuple(t[[0, 2, 3, 5]] for t in p))(after._project(drafts))
    after._attend(drafts[:4], [4])
    from bit_gemm_w4_amd import ops
    s = torch.arange(94).cuda()
    for a, b in zip(ops.kv_cache_read(layer.cache, s), ops.kv_cache_read(after.cache, s)):
        assert torch.equal(a, b)


def test_the_command_runs(mod, capsys):
    for args in (["--format", "int4"], ["--format", "fp8", "--window", "100", "--sinks", "4"]):
        mod.main(args)
    out = capsys.readouterr().out
    assert "lengths [707, 338]" in out and "lengths [704, 337]" in out


def test_refusals(mod):
    layer = _layer(mod, "int8", window=8)
    with pytest.raises(ValueError, match="full"):
        layer.extend(_rows(513, 4), [513])
    with pytest.raises(ValueError, match="no window"):
        layer.check(_rows(2, 4), [[-1, 0]])
