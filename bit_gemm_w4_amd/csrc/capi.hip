// capi.hip -- the exported C ABI (include/bitgemm.h): argument validation
// (fail-closed, "Low-precision LLM inference" §24 eligibility checklist and
// §31 fallback_policy) and kernel dispatch by M ("small batch and large
// prefill get different kernels", §24).  Validation touches no HIP API, so
// a rejected call never reaches the device.
#include <atomic>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/bitgemm.h"
#include "bg_internal.h"
#include "bg_kv.h"
#include "bg_overlap.h"

#define BG_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

thread_local char g_last_error[512] = "";
thread_local char g_last_kernel[160] = "";

void note_kernel(const char* name) {
    std::snprintf(g_last_kernel, sizeof(g_last_kernel), "%s", name ? name : "");
}

bg_status fail(bg_status st, const char* fmt, long long a = 0, long long b = 0) {
    std::snprintf(g_last_error, sizeof(g_last_error), fmt, a, b);
    return st;
}

// The same, with the entry point's name in front.
bg_status fail_in(const char* fn, bg_status st, const char* fmt, long long a = 0, long long b = 0) {
    const int n = std::snprintf(g_last_error, sizeof(g_last_error), "%s: ", fn);
    std::snprintf(g_last_error + n, sizeof(g_last_error) - n, fmt, a, b);
    return st;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bg_status launched(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) {
        std::snprintf(g_last_error, sizeof(g_last_error), "%s: launch failed: %s", what, hipGetErrorString(e));
        return BG_ERR_HIP;
    }
    g_last_error[0] = '\0';
    return BG_OK;
}

constexpr int64_t kMaxRows = int64_t(1) << 24;   // N, act_quant rows
constexpr int64_t kMaxDim = int64_t(1) << 20;    // K, cols
constexpr int64_t kMaxM = int64_t(65535) * 16;   // GEMM M: grid.y stays below 65536
constexpr int64_t kMaxGemvM = 256;               // explicit GEMV requests
constexpr int64_t kI8MaxKExcl = int64_t(1) << 17; // INT8 K bound: K * 2^14 < 2^31

// W4A16: small-M MFMA kernel up to kW4SkinnyMax rows, tiled MFMA kernel beyond;
// the VALU GEMV is selected explicitly only (BG_ALGO_GEMV).
constexpr int64_t kW4GemvMax = 0;
constexpr int64_t kW4SkinnyMax = 64;
constexpr int64_t kW8SkinnyMax = 32;

int w4_auto_algo(int64_t M, int64_t K) {
    if (K > bg::kW4DecodeMaxK) return BG_ALGO_TILED;
    if (M <= kW4GemvMax) return BG_ALGO_GEMV;
    if (M <= kW4SkinnyMax) return BG_ALGO_SKINNY;
    return BG_ALGO_TILED;
}

// W8A8: the small-M kernel streams the weights once per band of up to 64
// rows; the tiled kernel is flat in M until its 256 x 128 tiles fill the
// device. Measured on the 8B projection shapes: through M = 16 the small-M
// kernel (activations staged in LDS) wins on every shape, by 1.3-1.5x on the
// 28672-wide layer; above that the tiled grid wins once it has >= 128 tiles
// or M > 128, or M > 64 with a short K.
int w8_auto_algo(int64_t M, int64_t N, int64_t K) {
    if (M <= 16) return BG_ALGO_SKINNY;
    const int64_t tiles = ((M + 255) / 256) * ((N + 127) / 128);
    if (tiles >= 128 || M > 128) return BG_ALGO_TILED;
    if (M <= kW8SkinnyMax) return BG_ALGO_SKINNY;
    if (tiles < 48 && (M <= 64 || K >= 8192)) return BG_ALGO_SKINNY;
    return BG_ALGO_TILED;
}

// W8A8 with a workspace: the small-M kernel through M = 16, and through
// M = 32 on layers up to 4096 x 8192; beyond that the large-M kernel with K
// split wherever it measured faster than the small-M kernel on the
// projection shapes (N >= 6144, or K >= 8192, or M >= 32), else the choice
// above.
int w8_auto_algo_ws(int64_t M, int64_t N, int64_t K, int in_dtype, int a_gran) {
    if (M <= 16 || (M <= 32 && N <= 4096 && K <= 8192)) return BG_ALGO_SKINNY;
    bg::W8A8Args g{nullptr, nullptr, a_gran, nullptr, nullptr, 0, in_dtype == BG_FP8_E4M3, M, N, K, nullptr, BG_BF16};
    const bool fits = N >= 6144 || K >= 8192 || M >= 32;
    if (fits && bg::w8a8_tiled_split(g, true).S > 1) return BG_ALGO_TILED;
    return w8_auto_algo(M, N, K);
}

// Workspace bytes of a W4A16 kernel choice (0: none).
int64_t w4_ws_need(int algo, int64_t M, int64_t N, int64_t K) {
    if (algo == BG_ALGO_MID) return bg::w4a16_mid_workspace(M, N, K);
    if (algo != BG_ALGO_SPLITK) return 0;
    return M > kW4SkinnyMax ? bg::w4a16_gemm_split(M, N, K).ws_bytes : bg::w4a16_splitk_workspace(M, N, K);
}

// With a workspace, small M runs split-K where the small-M kernel's per-block
// re-staging of the activation rows costs more than split-K's cross-block
// reduction: from the measured crossovers (graph-replayed, cold weights) on
// the 4096/14336-wide projection shapes (N = 6144 and 4096 at K = 4096 stay
// on the small-M kernel through M = 16).
// Past the small-M range, split-K (of the large-M kernel) while its output
// tiles do not fill the device.
int w4_auto_algo_ws(int64_t M, int64_t N, int64_t K) {
    // mid-batch kernel: measured faster than the split small-M and the tiled
    // kernels on the projection shapes past M = 16 on the 28672-wide layer
    // (24.7 against 27.3 us at M = 24) and from M = 64 on the others, through
    // M = 128 (the tiled kernel wins again at M = 256)
    if (M <= 128 && (M >= 64 || (M > 16 && N >= 16384))) return BG_ALGO_MID;
    if (M > kW4SkinnyMax) return bg::w4a16_gemm_split(M, N, K).S > 1 ? BG_ALGO_SPLITK : BG_ALGO_TILED;
    // (measured: down, K = 14336, is faster split at every M >= 8; gate_up,
    // N = 28672, is faster unsplit through M = 16 -- 19.2-19.8 us against
    // 20.6-21.7 -- since the small-M kernel deals its tiles in one round)
    const bool split = (M >= 8 && K >= 8192) || (M > 16 && N > 4096) || M >= 24;
    if (split) return BG_ALGO_SPLITK;
    return K > bg::kW4DecodeMaxK ? BG_ALGO_TILED : BG_ALGO_SKINNY;
}

}  // namespace

BG_EXPORT bg_status w4_pack(const void* w, int w_dtype, int64_t N, int64_t K, int group, int asymmetric,
                            uint32_t* qweight, uint16_t* scales, uint8_t* zeros, void* stream) {
    if (!w || !qweight || !scales) return fail(BG_ERR_NULL, "w4_pack: w, qweight and scales must be non-NULL");
    if (asymmetric && !zeros) return fail(BG_ERR_NULL, "w4_pack: asymmetric packing needs a zeros buffer");
    if (!asymmetric && zeros) return fail(BG_ERR_UNSUPPORTED, "w4_pack: zeros must be NULL when symmetric");
    if (w_dtype != BG_F32 && w_dtype != BG_F16 && w_dtype != BG_BF16)
        return fail(BG_ERR_DTYPE, "w4_pack: w_dtype %lld is not F32/F16/BF16", w_dtype);
    if (group != 128) return fail(BG_ERR_UNSUPPORTED, "w4_pack: group %lld (only 128 is supported)", group);
    if (N < 16 || N > kMaxRows || N % 16) return fail(BG_ERR_SHAPE, "w4_pack: N=%lld must be a multiple of 16", N);
    if (K < 256 || K > kMaxDim || K % 256) return fail(BG_ERR_SHAPE, "w4_pack: K=%lld must be a multiple of 256", K);
    if (N * (K / 8) / 256 >= (int64_t(1) << 31)) return fail(BG_ERR_SHAPE, "w4_pack: N*K=%lld too large", N * K);
    if (!aligned16(w) || !aligned16(qweight) || !aligned16(scales) || (zeros && !aligned16(zeros)))
        return fail(BG_ERR_ALIGN, "w4_pack: pointers must be 16-byte aligned");
    note_kernel(bg::launch_w4_pack(w, w_dtype, N, K, asymmetric != 0, qweight, scales, zeros,
                       static_cast<hipStream_t>(stream)));
    return launched("w4_pack");
}

BG_EXPORT int gemm_w4a16_algo(int64_t M, int64_t N, int64_t K, int x_dtype) {
    (void)N; (void)x_dtype;
    return w4_auto_algo(M, K);
}

static bg_status w4a16_impl(const void* x, int x_dtype, int64_t M, int64_t K, const uint32_t* qweight,
                            const uint16_t* scales, const uint8_t* zeros, int64_t N, int group, void* y,
                            void* ws, int64_t ws_bytes, bool with_ws, int algo, void* stream) {
    if (!x || !qweight || !scales || !y) return fail(BG_ERR_NULL, "gemm_w4a16: x, qweight, scales and y must be non-NULL");
    if (x_dtype != BG_F16 && x_dtype != BG_BF16)
        return fail(BG_ERR_DTYPE, "gemm_w4a16: x_dtype %lld is not F16/BF16", x_dtype);
    if (group != 128) return fail(BG_ERR_UNSUPPORTED, "gemm_w4a16: group %lld (only 128 is supported)", group);
    if (M < 1 || M > kMaxM) return fail(BG_ERR_SHAPE, "gemm_w4a16: M=%lld out of range", M);
    if (N < 16 || N > kMaxRows || N % 16) return fail(BG_ERR_SHAPE, "gemm_w4a16: N=%lld must be a multiple of 16", N);
    if (K < 256 || K > kMaxDim || K % 256) return fail(BG_ERR_SHAPE, "gemm_w4a16: K=%lld must be a multiple of 256", K);
    if (!aligned16(x) || !aligned16(qweight) || !aligned16(scales) || !aligned16(y) || (zeros && !aligned16(zeros)) ||
        (ws && !aligned16(ws)))
        return fail(BG_ERR_ALIGN, "gemm_w4a16: pointers must be 16-byte aligned");
    if (algo == BG_ALGO_AUTO) algo = with_ws ? w4_auto_algo_ws(M, N, K) : w4_auto_algo(M, K);
    if (algo == BG_ALGO_GEMV && (M > kMaxGemvM || !bg::w4a16_gemv_supported(M, K)))
        return fail(BG_ERR_SHAPE, "gemm_w4a16: the GEMV kernel takes M <= 256 and K <= 18432 (M=%lld, K=%lld)", M, K);
    if (algo == BG_ALGO_SKINNY && K > bg::kW4DecodeMaxK)
        return fail(BG_ERR_SHAPE, "gemm_w4a16: the small-M kernel takes K <= 65536 (K=%lld)", K);
    if (algo == BG_ALGO_SPLITK && !with_ws)
        return fail(BG_ERR_WORKSPACE, "gemm_w4a16: the split-K kernels need gemm_w4a16_ws");
    if (with_ws && (algo == BG_ALGO_SPLITK || algo == BG_ALGO_MID)) {
        const int64_t need = w4_ws_need(algo, M, N, K);
        if (need > 0 && (!ws || ws_bytes < need))
            return fail(BG_ERR_WORKSPACE, "gemm_w4a16: workspace of %lld bytes needed (got %lld)", need, ws ? ws_bytes : 0);
    }
    const bool bf16 = x_dtype == BG_BF16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (algo) {
        case BG_ALGO_GEMV: note_kernel(bg::launch_w4a16_gemv(x, bf16, M, K, qweight, scales, zeros, N, y, s)); break;
        case BG_ALGO_SKINNY: note_kernel(bg::launch_w4a16_skinny(x, bf16, M, K, qweight, scales, zeros, N, y, s)); break;
        case BG_ALGO_TILED: note_kernel(bg::launch_w4a16_tiled(x, bf16, M, K, qweight, scales, zeros, N, y, s)); break;
        case BG_ALGO_MID:
            note_kernel(bg::launch_w4a16_mid(x, bf16, M, K, qweight, scales, zeros, N, y, with_ws ? ws : nullptr, s));
            break;
        case BG_ALGO_SPLITK:
            if (M > kW4SkinnyMax)
                note_kernel(bg::launch_w4a16_gemm(x, bf16, M, K, qweight, scales, zeros, N, y, ws, s));
            else
                note_kernel(bg::launch_w4a16_splitk(x, bf16, M, K, qweight, scales, zeros, N, y, ws, s));
            break;
        default: return fail(BG_ERR_UNSUPPORTED, "gemm_w4a16: unknown algo %lld", algo);
    }
    return launched("gemm_w4a16");
}

BG_EXPORT bg_status gemm_w4a16_ex(const void* x, int x_dtype, int64_t M, int64_t K, const uint32_t* qweight,
                                  const uint16_t* scales, const uint8_t* zeros, int64_t N, int group, void* y,
                                  int algo, void* stream) {
    return w4a16_impl(x, x_dtype, M, K, qweight, scales, zeros, N, group, y, nullptr, 0, false, algo, stream);
}

BG_EXPORT bg_status gemm_w4a16_ws(const void* x, int x_dtype, int64_t M, int64_t K, const uint32_t* qweight,
                                  const uint16_t* scales, const uint8_t* zeros, int64_t N, int group, void* y,
                                  void* workspace, int64_t workspace_bytes, int algo, void* stream) {
    return w4a16_impl(x, x_dtype, M, K, qweight, scales, zeros, N, group, y, workspace, workspace_bytes, true, algo,
                      stream);
}

BG_EXPORT int64_t gemm_w4a16_workspace_bytes(int64_t M, int64_t N, int64_t K, int algo) {
    if (M < 1 || M > kMaxM || N < 16 || N % 16 || K < 256 || K % 256) return 0;
    if (algo == BG_ALGO_AUTO) algo = w4_auto_algo_ws(M, N, K);
    return w4_ws_need(algo, M, N, K);
}

BG_EXPORT bg_status gemm_w4a16(const void* x, int x_dtype, int64_t M, int64_t K, const uint32_t* qweight,
                               const uint16_t* scales, const uint8_t* zeros, int64_t N, int group, void* y,
                               void* stream) {
    return gemm_w4a16_ex(x, x_dtype, M, K, qweight, scales, zeros, N, group, y, BG_ALGO_AUTO, stream);
}

// ---- gemm_w4a16_noalloc: split-K partials in a static device array ----
//
// For callers that cannot allocate (code under HIP graph capture, serving
// loops, harnesses that forbid hipMalloc).  `scratch` lives in the code
// object: every GPU that runs the library holds its own copy, at its own
// address, until the process ends.  Host code never passes the array's name
// to a kernel (on the host it is only a stand-in for the symbol); it uses the
// device address hipGetSymbolAddress returns, looked up once per device with
// that device current.
static __device__ __align__(256) uint8_t scratch[BG_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
std::atomic<void*> g_scratch_ptr[kMaxDevices];

bg_status hip_fail(const char* what, hipError_t e) {
    std::snprintf(g_last_error, sizeof(g_last_error), "gemm_w4a16_noalloc: %s: %s", what, hipGetErrorString(e));
    return BG_ERR_HIP;
}

// Device address of `scratch` on the device `stream` runs on, which must be
// the current device.
bg_status scratch_address(void* stream, void** out) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail("hipGetDevice", e);
    if (dev < 0 || dev >= kMaxDevices) return fail(BG_ERR_UNSUPPORTED, "gemm_w4a16_noalloc: device %lld out of range", dev);
    if (stream) {
        hipDevice_t sdev = -1;
        e = hipStreamGetDevice(static_cast<hipStream_t>(stream), &sdev);
        if (e != hipSuccess) return hip_fail("hipStreamGetDevice", e);
        if (sdev != dev)
            return fail(BG_ERR_UNSUPPORTED, "gemm_w4a16_noalloc: the stream is on device %lld, the current device is %lld",
                        sdev, dev);
    }
    void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
    if (!p) {
        std::lock_guard<std::mutex> lk(g_scratch_mu);
        p = g_scratch_ptr[dev].load(std::memory_order_relaxed);
        if (!p) {
            e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
            if (e != hipSuccess || !p) return hip_fail("hipGetSymbolAddress(scratch)", e);
            g_scratch_ptr[dev].store(p, std::memory_order_release);
        }
    }
    *out = p;
    return BG_OK;
}

}  // namespace

BG_EXPORT bg_status gemm_w4a16_noalloc(const void* x, int x_dtype, int64_t M, int64_t K, const uint32_t* qweight,
                                       const uint16_t* scales, const uint8_t* zeros, int64_t N, int group, void* y,
                                       void* stream) {
    // the shape checks of gemm_w4a16 come first, so the size asked of the
    // scratch is only computed for an eligible call
    if (!x || !qweight || !scales || !y) return fail(BG_ERR_NULL, "gemm_w4a16: x, qweight, scales and y must be non-NULL");
    if (M < 1 || M > kMaxM) return fail(BG_ERR_SHAPE, "gemm_w4a16: M=%lld out of range", M);
    if (N < 16 || N > kMaxRows || N % 16) return fail(BG_ERR_SHAPE, "gemm_w4a16: N=%lld must be a multiple of 16", N);
    if (K < 256 || K > kMaxDim || K % 256) return fail(BG_ERR_SHAPE, "gemm_w4a16: K=%lld must be a multiple of 256", K);
    const int algo = w4_auto_algo_ws(M, N, K);
    const int64_t need = w4_ws_need(algo, M, N, K);
    if (need > BG_NOALLOC_SCRATCH_BYTES)
        return fail(BG_ERR_WORKSPACE,
                    "gemm_w4a16_noalloc: this shape needs %lld bytes of scratch; the static scratch holds %lld "
                    "(use gemm_w4a16_ws with a larger workspace)",
                    need, (long long)BG_NOALLOC_SCRATCH_BYTES);
    void* ws = nullptr;
    if (need > 0) {
        const bg_status st = scratch_address(stream, &ws);
        if (st != BG_OK) return st;
    }
    return w4a16_impl(x, x_dtype, M, K, qweight, scales, zeros, N, group, y, ws, need, true, algo, stream);
}

static bg_status act_quant(const char* name, bool fp8, const void* x, int x_dtype, int64_t rows, int64_t cols,
                           int gran, const float* col_mul, bool smooth, void* q, float* scales, void* stream) {
    if (!x || !q || !scales) return fail(BG_ERR_NULL, "act_quant: x, q and scales must be non-NULL");
    if (smooth && !col_mul) return fail(BG_ERR_NULL, "act_quant: col_mul must be non-NULL");
    if (x_dtype != BG_F32 && x_dtype != BG_F16 && x_dtype != BG_BF16)
        return fail(BG_ERR_DTYPE, "act_quant: x_dtype %lld is not F32/F16/BF16", x_dtype);
    if (gran < BG_GRAN_TENSOR || gran > BG_GRAN_BLOCK128)
        return fail(BG_ERR_UNSUPPORTED, "act_quant: unknown granularity %lld", gran);
    if (rows < 1 || rows > kMaxRows) return fail(BG_ERR_SHAPE, "act_quant: rows=%lld out of range", rows);
    if (cols < 128 || cols > kMaxDim || cols % 128)
        return fail(BG_ERR_SHAPE, "act_quant: cols=%lld must be a multiple of 128", cols);
    if (gran == BG_GRAN_BLOCK128 && rows % 128)
        return fail(BG_ERR_SHAPE, "act_quant: BLOCK128 needs rows %% 128 == 0 (rows=%lld)", rows);
    if (!aligned16(x) || !aligned16(q) || !aligned16(scales) || (col_mul && !aligned16(col_mul)))
        return fail(BG_ERR_ALIGN, "act_quant: pointers must be 16-byte aligned");
    note_kernel(bg::launch_act_quant(x, x_dtype, rows, cols, gran, fp8, q, scales, smooth ? col_mul : nullptr,
                                     static_cast<hipStream_t>(stream)));
    return launched(name);
}

BG_EXPORT bg_status act_quant_int8(const void* x, int x_dtype, int64_t rows, int64_t cols, int gran, int8_t* q,
                                   float* scales, void* stream) {
    return act_quant("act_quant_int8", false, x, x_dtype, rows, cols, gran, nullptr, false, q, scales, stream);
}

BG_EXPORT bg_status act_quant_fp8(const void* x, int x_dtype, int64_t rows, int64_t cols, int gran, uint8_t* q,
                                  float* scales, void* stream) {
    return act_quant("act_quant_fp8", true, x, x_dtype, rows, cols, gran, nullptr, false, q, scales, stream);
}

BG_EXPORT bg_status act_quant_int8_smooth(const void* x, int x_dtype, int64_t rows, int64_t cols, int gran,
                                          const float* col_mul, int8_t* q, float* scales, void* stream) {
    return act_quant("act_quant_int8_smooth", false, x, x_dtype, rows, cols, gran, col_mul, true, q, scales, stream);
}

BG_EXPORT bg_status act_quant_fp8_smooth(const void* x, int x_dtype, int64_t rows, int64_t cols, int gran,
                                         const float* col_mul, uint8_t* q, float* scales, void* stream) {
    return act_quant("act_quant_fp8_smooth", true, x, x_dtype, rows, cols, gran, col_mul, true, q, scales, stream);
}

static bg_status act_quant_mx(const char* fn, bool fp4, const void* x, int x_dtype, int64_t rows, int64_t cols,
                              uint8_t* q, uint8_t* e8m0, void* stream) {
    if (!x || !q || !e8m0) return fail_in(fn, BG_ERR_NULL, "x, q and e8m0 must be non-NULL");
    if (x_dtype != BG_F32 && x_dtype != BG_F16 && x_dtype != BG_BF16)
        return fail_in(fn, BG_ERR_DTYPE, "x_dtype %lld is not F32/F16/BF16", x_dtype);
    if (rows < 1 || rows > kMaxRows) return fail_in(fn, BG_ERR_SHAPE, "rows=%lld out of range", rows);
    if (cols < 32 || cols > kMaxDim || cols % 32)
        return fail_in(fn, BG_ERR_SHAPE, "cols=%lld must be a multiple of 32", cols);
    if (!aligned16(x) || !aligned16(q)) return fail_in(fn, BG_ERR_ALIGN, "x and q must be 16-byte aligned");
    note_kernel(bg::launch_quant_mx32(x, x_dtype, rows, cols, fp4, q, e8m0, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

BG_EXPORT bg_status act_quant_mxfp8(const void* x, int x_dtype, int64_t rows, int64_t cols, uint8_t* q,
                                    uint8_t* e8m0, void* stream) {
    return act_quant_mx("act_quant_mxfp8", false, x, x_dtype, rows, cols, q, e8m0, stream);
}

BG_EXPORT bg_status act_quant_mxfp4(const void* x, int x_dtype, int64_t rows, int64_t cols, uint8_t* q,
                                    uint8_t* e8m0, void* stream) {
    return act_quant_mx("act_quant_mxfp4", true, x, x_dtype, rows, cols, q, e8m0, stream);
}

// K granularity: one pair of 64-byte stages, i.e. 128 MXFP8 or 256 MXFP4 elements.
static bg_status gemm_mx(const char* fn, bool fp4, const uint8_t* a, const uint8_t* a_e8m0, const uint8_t* w,
                         const uint8_t* w_e8m0, int64_t M, int64_t N, int64_t K, void* y, int out_dtype,
                         void* stream) {
    if (!a || !a_e8m0 || !w || !w_e8m0 || !y)
        return fail_in(fn, BG_ERR_NULL, "a, a_e8m0, w, w_e8m0 and y must be non-NULL");
    if (out_dtype != BG_BF16 && out_dtype != BG_F16 && out_dtype != BG_F32)
        return fail_in(fn, BG_ERR_DTYPE, "out_dtype %lld is not BF16/F16/F32", out_dtype);
    const int64_t kq = fp4 ? 256 : 128;
    const int64_t row_bytes = fp4 ? K / 2 : K;
    if (M < 1 || M > kMaxM) return fail_in(fn, BG_ERR_SHAPE, "M=%lld out of range", M);
    if (N < 16 || N > kMaxRows || N % 16) return fail_in(fn, BG_ERR_SHAPE, "N=%lld must be a multiple of 16", N);
    if (K < kq || K > kMaxDim || K % kq)
        return fail_in(fn, BG_ERR_SHAPE, "K=%lld must be a multiple of %lld", K, kq);
    if (M * row_bytes >= (int64_t(1) << 31) || N * row_bytes >= (int64_t(1) << 31))
        return fail_in(fn, BG_ERR_SHAPE, "the A and W operands must each be below 2^31 bytes");
    if (!aligned16(a) || !aligned16(w) || !aligned16(y) || !aligned16(a_e8m0) || !aligned16(w_e8m0))
        return fail_in(fn, BG_ERR_ALIGN, "pointers must be 16-byte aligned");
    const int gran = fp4 ? 5 : 4;
    bg::W8A8Args g{a, reinterpret_cast<const float*>(a_e8m0), gran, w, reinterpret_cast<const float*>(w_e8m0), gran,
                   true, M, N, K, y, out_dtype};
    note_kernel(bg::launch_w8a8_tiled(g, nullptr, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

BG_EXPORT bg_status gemm_mxfp8(const uint8_t* a, const uint8_t* a_e8m0, const uint8_t* w, const uint8_t* w_e8m0,
                               int64_t M, int64_t N, int64_t K, void* y, int out_dtype, void* stream) {
    return gemm_mx("gemm_mxfp8", false, a, a_e8m0, w, w_e8m0, M, N, K, y, out_dtype, stream);
}

BG_EXPORT bg_status gemm_mxfp4(const uint8_t* a, const uint8_t* a_e8m0, const uint8_t* w, const uint8_t* w_e8m0,
                               int64_t M, int64_t N, int64_t K, void* y, int out_dtype, void* stream) {
    return gemm_mx("gemm_mxfp4", true, a, a_e8m0, w, w_e8m0, M, N, K, y, out_dtype, stream);
}

BG_EXPORT int gemm_w8a8_algo(int64_t M, int64_t N, int64_t K, int in_dtype) {
    (void)in_dtype;
    return w8_auto_algo(M, N, K);
}

static bg_status w8a8_impl(const void* a, const float* a_scales, int a_gran, const void* w, const float* w_scales,
                           int w_gran, int in_dtype, int64_t M, int64_t N, int64_t K, void* y, int out_dtype,
                           void* ws, int64_t ws_bytes, bool with_ws, int algo, void* stream) {
    if (!a || !w || !y) return fail(BG_ERR_NULL, "gemm_w8a8: a, w and y must be non-NULL");
    if (in_dtype != BG_I8 && in_dtype != BG_FP8_E4M3)
        return fail(BG_ERR_DTYPE, "gemm_w8a8: in_dtype %lld is not I8/FP8_E4M3", in_dtype);
    const bool raw = out_dtype == BG_I32;
    if (raw && in_dtype != BG_I8) return fail(BG_ERR_DTYPE, "gemm_w8a8: I32 output needs I8 inputs");
    if (!raw && out_dtype != BG_BF16 && out_dtype != BG_F16 && out_dtype != BG_F32)
        return fail(BG_ERR_DTYPE, "gemm_w8a8: out_dtype %lld is not BF16/F16/F32/I32", out_dtype);
    if (!raw && (!a_scales || !w_scales)) return fail(BG_ERR_NULL, "gemm_w8a8: scales must be non-NULL");
    const bool per = (a_gran == BG_GRAN_TENSOR || a_gran == BG_GRAN_ROW) &&
                     (w_gran == BG_GRAN_TENSOR || w_gran == BG_GRAN_ROW);
    const bool block = a_gran == BG_GRAN_ROW_G128 && w_gran == BG_GRAN_BLOCK128;
    if (!raw && !per && !(block && in_dtype == BG_FP8_E4M3))
        return fail(BG_ERR_UNSUPPORTED, "gemm_w8a8: granularity pair (%lld, %lld) not supported", a_gran, w_gran);
    if (M < 1 || M > kMaxM) return fail(BG_ERR_SHAPE, "gemm_w8a8: M=%lld out of range", M);
    if (N < 16 || N > kMaxRows || N % 16) return fail(BG_ERR_SHAPE, "gemm_w8a8: N=%lld must be a multiple of 16", N);
    if (K < 128 || K > kMaxDim || K % 128) return fail(BG_ERR_SHAPE, "gemm_w8a8: K=%lld must be a multiple of 128", K);
    // |acc| <= K * 128 * 128 must stay below 2^31: K <= 130944 (K = 131072
    // with every code at -128 would reach exactly 2^31 and wrap)
    if (in_dtype == BG_I8 && K >= kI8MaxKExcl)
        return fail(BG_ERR_SHAPE, "gemm_w8a8: K=%lld too long for exact INT32 accumulation (K < 131072)", K);
    if (block && N % 128) return fail(BG_ERR_SHAPE, "gemm_w8a8: BLOCK128 weights need N %% 128 == 0 (N=%lld)", N);
    if (!aligned16(a) || !aligned16(w) || !aligned16(y) || (a_scales && !aligned16(a_scales)) ||
        (w_scales && !aligned16(w_scales)) || (ws && !aligned16(ws)))
        return fail(BG_ERR_ALIGN, "gemm_w8a8: pointers must be 16-byte aligned");
    if (algo == BG_ALGO_AUTO) algo = with_ws ? w8_auto_algo_ws(M, N, K, in_dtype, a_gran) : w8_auto_algo(M, N, K);
    bg::W8A8Args g{a, a_scales, raw ? BG_GRAN_ROW : a_gran, w, w_scales, raw ? BG_GRAN_ROW : w_gran,
                   in_dtype == BG_FP8_E4M3, M, N, K, y, out_dtype};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (algo == BG_ALGO_TILED && with_ws) {
        const int64_t need = bg::w8a8_tiled_split(g, true).ws_bytes;
        if (need > 0 && (!ws || ws_bytes < need))
            return fail(BG_ERR_WORKSPACE, "gemm_w8a8: workspace of %lld bytes needed (got %lld)", need, ws ? ws_bytes : 0);
    }
    switch (algo) {
        case BG_ALGO_SKINNY: note_kernel(bg::launch_w8a8_skinny(g, s)); break;
        case BG_ALGO_TILED: note_kernel(bg::launch_w8a8_tiled(g, with_ws ? ws : nullptr, s)); break;
        default: return fail(BG_ERR_UNSUPPORTED, "gemm_w8a8: unknown algo %lld", algo);
    }
    return launched("gemm_w8a8");
}

BG_EXPORT bg_status gemm_w8a8_ex(const void* a, const float* a_scales, int a_gran, const void* w,
                                 const float* w_scales, int w_gran, int in_dtype, int64_t M, int64_t N, int64_t K,
                                 void* y, int out_dtype, int algo, void* stream) {
    return w8a8_impl(a, a_scales, a_gran, w, w_scales, w_gran, in_dtype, M, N, K, y, out_dtype, nullptr, 0, false,
                     algo, stream);
}

BG_EXPORT bg_status gemm_w8a8_ws(const void* a, const float* a_scales, int a_gran, const void* w,
                                 const float* w_scales, int w_gran, int in_dtype, int64_t M, int64_t N, int64_t K,
                                 void* y, int out_dtype, void* workspace, int64_t workspace_bytes, int algo,
                                 void* stream) {
    return w8a8_impl(a, a_scales, a_gran, w, w_scales, w_gran, in_dtype, M, N, K, y, out_dtype, workspace,
                     workspace_bytes, true, algo, stream);
}

BG_EXPORT int64_t gemm_w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K, int in_dtype, int a_gran, int algo) {
    if (M < 1 || M > kMaxM || N < 16 || N > kMaxRows || N % 16 || K < 128 || K > kMaxDim || K % 128) return 0;
    if (algo == BG_ALGO_AUTO) algo = w8_auto_algo_ws(M, N, K, in_dtype, a_gran);
    if (algo != BG_ALGO_TILED) return 0;
    bg::W8A8Args g{nullptr, nullptr, a_gran, nullptr, nullptr, 0, in_dtype == BG_FP8_E4M3, M, N, K, nullptr, BG_BF16};
    return bg::w8a8_tiled_split(g, true).ws_bytes;
}

BG_EXPORT bg_status gemm_w8a8(const void* a, const float* a_scales, int a_gran, const void* w,
                              const float* w_scales, int w_gran, int in_dtype, int64_t M, int64_t N, int64_t K,
                              void* y, int out_dtype, void* stream) {
    return gemm_w8a8_ex(a, a_scales, a_gran, w, w_scales, w_gran, in_dtype, M, N, K, y, out_dtype, BG_ALGO_AUTO,
                        stream);
}

// ---- LLM.int8() outlier side path ----

BG_EXPORT int64_t act_quant_outlier_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows < 1 || rows > kMaxRows || cols < 128 || cols > kMaxDim || cols % 128) return 0;
    return bg::outlier_ws_bytes(rows, cols);
}

BG_EXPORT bg_status act_quant_int8_outlier(const void* x, int x_dtype, int64_t rows, int64_t cols, float tau,
                                           int8_t* q, float* scales, int32_t* idx, int32_t* count, void* workspace,
                                           int64_t workspace_bytes, void* stream) {
    const char* fn = "act_quant_int8_outlier";
    if (!x || !q || !scales || !idx || !count || !workspace)
        return fail_in(fn, BG_ERR_NULL, "x, q, scales, idx, count and workspace must be non-NULL");
    if (x_dtype != BG_F32 && x_dtype != BG_F16 && x_dtype != BG_BF16)
        return fail_in(fn, BG_ERR_DTYPE, "x_dtype %lld is not F32/F16/BF16", x_dtype);
    if (tau != tau) return fail_in(fn, BG_ERR_UNSUPPORTED, "tau is NaN");
    if (rows < 1 || rows > kMaxRows) return fail_in(fn, BG_ERR_SHAPE, "rows=%lld out of range", rows);
    if (cols < 128 || cols > kMaxDim || cols % 128)
        return fail_in(fn, BG_ERR_SHAPE, "cols=%lld must be a multiple of 128", cols);
    const int64_t need = bg::outlier_ws_bytes(rows, cols);
    if (workspace_bytes < need)
        return fail_in(fn, BG_ERR_WORKSPACE, "workspace of %lld bytes needed (got %lld)", need, workspace_bytes);
    if (!aligned16(x) || !aligned16(q) || !aligned16(scales) || !aligned16(workspace) ||
        (reinterpret_cast<uintptr_t>(idx) & 3u) || (reinterpret_cast<uintptr_t>(count) & 3u))
        return fail_in(fn, BG_ERR_ALIGN, "x, q, scales and workspace must be 16-byte aligned, idx and count 4-byte");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const float* mask = nullptr;
    bg::launch_outlier_detect(x, x_dtype, rows, cols, tau, static_cast<float*>(workspace), idx, count, &mask, s);
    note_kernel(bg::launch_act_quant(x, x_dtype, rows, cols, BG_GRAN_ROW, false, q, scales, mask, s));
    return launched(fn);
}

BG_EXPORT bg_status gemm_w8a8_outlier(const int8_t* a, const float* a_scales, const int8_t* w, const float* w_scales,
                                      int w_gran, const void* x, int x_dtype, const int32_t* idx,
                                      const int32_t* count, int64_t M, int64_t N, int64_t K, void* y, int out_dtype,
                                      void* stream) {
    const char* fn = "gemm_w8a8_outlier";
    if (!a || !a_scales || !w || !w_scales || !x || !idx || !count || !y)
        return fail_in(fn, BG_ERR_NULL, "a, a_scales, w, w_scales, x, idx, count and y must be non-NULL");
    if (w_gran != BG_GRAN_TENSOR && w_gran != BG_GRAN_ROW)
        return fail_in(fn, BG_ERR_UNSUPPORTED, "w_gran %lld is not TENSOR/ROW", w_gran);
    if (x_dtype != BG_F32 && x_dtype != BG_F16 && x_dtype != BG_BF16)
        return fail_in(fn, BG_ERR_DTYPE, "x_dtype %lld is not F32/F16/BF16", x_dtype);
    if (out_dtype != BG_BF16 && out_dtype != BG_F16 && out_dtype != BG_F32)
        return fail_in(fn, BG_ERR_DTYPE, "out_dtype %lld is not BF16/F16/F32", out_dtype);
    if (M < 1 || M > kMaxM) return fail_in(fn, BG_ERR_SHAPE, "M=%lld out of range", M);
    if (N < 16 || N > kMaxRows || N % 16) return fail_in(fn, BG_ERR_SHAPE, "N=%lld must be a multiple of 16", N);
    if (K < 128 || K >= kI8MaxKExcl || K % 128)
        return fail_in(fn, BG_ERR_SHAPE, "K=%lld must be a multiple of 128 and below 131072", K);
    if (!aligned16(a) || !aligned16(w) || !aligned16(y) || !aligned16(a_scales) || !aligned16(w_scales) ||
        (reinterpret_cast<uintptr_t>(x) & 3u) || (reinterpret_cast<uintptr_t>(idx) & 3u) ||
        (reinterpret_cast<uintptr_t>(count) & 3u))
        return fail_in(fn, BG_ERR_ALIGN, "a, w, y and the scales must be 16-byte aligned, x, idx and count 4-byte");
    bg::W8A8Args g{a, a_scales, BG_GRAN_ROW, w, w_scales, w_gran, false, M, N, K, y, out_dtype};
    g.ox = x;
    g.ox_dt = x_dtype;
    g.oidx = idx;
    g.ocnt = count;
    note_kernel(bg::launch_w8a8_tiled(g, nullptr, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

static bg_status w4a8_impl(const int8_t* a, const float* a_scales, int a_gran, int64_t M, int64_t K,
                           const uint32_t* qweight, const uint16_t* scales, const uint8_t* zeros, int64_t N, int group,
                           void* y, int out_dtype, void* ws, int64_t ws_bytes, bool with_ws, void* stream) {
    if (!a || !a_scales || !qweight || !scales || !y)
        return fail(BG_ERR_NULL, "gemm_w4a8: a, a_scales, qweight, scales and y must be non-NULL");
    if (a_gran != BG_GRAN_TENSOR && a_gran != BG_GRAN_ROW)
        return fail(BG_ERR_UNSUPPORTED, "gemm_w4a8: a_gran %lld is not TENSOR/ROW", a_gran);
    if (out_dtype != BG_BF16 && out_dtype != BG_F16 && out_dtype != BG_F32)
        return fail(BG_ERR_DTYPE, "gemm_w4a8: out_dtype %lld is not BF16/F16/F32", out_dtype);
    if (group != 128) return fail(BG_ERR_UNSUPPORTED, "gemm_w4a8: group %lld (only 128 is supported)", group);
    if (M < 1 || M > kMaxM) return fail(BG_ERR_SHAPE, "gemm_w4a8: M=%lld out of range", M);
    if (N < 16 || N > kMaxRows || N % 16) return fail(BG_ERR_SHAPE, "gemm_w4a8: N=%lld must be a multiple of 16", N);
    if (K < 256 || K > kMaxDim || K % 256) return fail(BG_ERR_SHAPE, "gemm_w4a8: K=%lld must be a multiple of 256", K);
    if (M * K >= (int64_t(1) << 31)) return fail(BG_ERR_SHAPE, "gemm_w4a8: M*K=%lld too large", M * K);
    if (!aligned16(a) || !aligned16(a_scales) || !aligned16(qweight) || !aligned16(scales) || !aligned16(y) ||
        (zeros && !aligned16(zeros)) || (ws && !aligned16(ws)))
        return fail(BG_ERR_ALIGN, "gemm_w4a8: pointers must be 16-byte aligned");
    if (bg::w4a8_decode_fits(M, N, K)) {
        note_kernel(bg::launch_w4a8_decode(a, a_scales, a_gran == BG_GRAN_ROW, M, K, qweight, scales, zeros, N, y,
                                           out_dtype, static_cast<hipStream_t>(stream)));
        return launched("gemm_w4a8");
    }
    void* use_ws = nullptr;
    if (with_ws) {
        const int64_t need = bg::w4a8_gemm_split(M, N, K).ws_bytes;
        if (need > 0) {
            if (!ws || ws_bytes < need)
                return fail(BG_ERR_WORKSPACE, "gemm_w4a8: workspace of %lld bytes needed (got %lld)", need,
                            ws ? ws_bytes : 0);
            use_ws = ws;
        }
    }
    note_kernel(bg::launch_w4a8_gemm(a, a_scales, a_gran == BG_GRAN_ROW, M, K, qweight, scales, zeros, N, y,
                                     out_dtype, use_ws, static_cast<hipStream_t>(stream)));
    return launched("gemm_w4a8");
}

BG_EXPORT bg_status gemm_w4a8(const int8_t* a, const float* a_scales, int a_gran, int64_t M, int64_t K,
                              const uint32_t* qweight, const uint16_t* scales, const uint8_t* zeros, int64_t N,
                              int group, void* y, int out_dtype, void* stream) {
    return w4a8_impl(a, a_scales, a_gran, M, K, qweight, scales, zeros, N, group, y, out_dtype, nullptr, 0, false,
                     stream);
}

BG_EXPORT bg_status gemm_w4a8_ws(const int8_t* a, const float* a_scales, int a_gran, int64_t M, int64_t K,
                                 const uint32_t* qweight, const uint16_t* scales, const uint8_t* zeros, int64_t N,
                                 int group, void* y, int out_dtype, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
    return w4a8_impl(a, a_scales, a_gran, M, K, qweight, scales, zeros, N, group, y, out_dtype, workspace,
                     workspace_bytes, true, stream);
}

BG_EXPORT int64_t gemm_w4a8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || M > kMaxM || N < 16 || N > kMaxRows || N % 16 || K < 256 || K > kMaxDim || K % 256) return 0;
    if (bg::w4a8_decode_fits(M, N, K)) return 0;
    return bg::w4a8_gemm_split(M, N, K).ws_bytes;
}

// ---- quantized KV cache ----

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int kMaxKvHeads = 1024;
constexpr int64_t kMaxBatch = 65535;             // attention: grid.z

// The cache descriptor of `fn`, checked.
bg_status kv_cache_of(const char* fn, const bg_kv_cache* c, bg::KvCache* out) {
    if (!c) return fail_in(fn, BG_ERR_NULL, "cache must be non-NULL");
    if (!c->k || !c->v || !c->k_scales || !c->v_scales)
        return fail_in(fn, BG_ERR_NULL, "the cache's k, v, k_scales and v_scales must be non-NULL");
    if (c->format != BG_I8 && c->format != BG_FP8_E4M3 && c->format != BG_U4)
        return fail_in(fn, BG_ERR_DTYPE, "cache format %lld is not I8/FP8_E4M3/U4", c->format);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail_in(fn, BG_ERR_SHAPE, "head_dim %lld is not 64, 128 or 256", c->head_dim);
    if (c->kv_heads < 1 || c->kv_heads > kMaxKvHeads)
        return fail_in(fn, BG_ERR_SHAPE, "kv_heads %lld out of range", c->kv_heads);
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return fail_in(fn, BG_ERR_SHAPE, "page_size %lld is not a power of two in 16..1024", c->page_size);
    if (c->pages < 1 || c->pages > INT32_MAX) return fail_in(fn, BG_ERR_SHAPE, "pages %lld out of range", c->pages);
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scales) || !aligned16(c->v_scales))
        return fail_in(fn, BG_ERR_ALIGN, "the cache's buffers must be 16-byte aligned");
    *out = bg::KvCache{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), static_cast<uint32_t*>(c->k_scales),
                       static_cast<uint32_t*>(c->v_scales), c->pages, __builtin_ctz((unsigned)c->page_size),
                       c->kv_heads, c->head_dim, c->format};
    return BG_OK;
}

// The sizes of p, checked; with `pointers`, what a launch reads too.
bg_status kv_attn_args(const char* fn, const bg_kv_attn* p, bool tree, bool pointers, bg::KvAttnArgs* a) {
    if (!p) return fail_in(fn, BG_ERR_NULL, "args must be non-NULL");
    const bg_status st = kv_cache_of(fn, p->cache, &a->c);
    if (st != BG_OK) return st;
    if (p->dtype != BG_F16 && p->dtype != BG_BF16) return fail_in(fn, BG_ERR_DTYPE, "dtype %lld is not F16/BF16", p->dtype);
    if (p->tokens < 0 || p->tokens > kMaxTokens) return fail_in(fn, BG_ERR_SHAPE, "tokens=%lld out of range", p->tokens);
    if (p->tokens * (p->q_heads > 0 ? p->q_heads : 0) > (int64_t(1) << 28))
        return fail_in(fn, BG_ERR_SHAPE, "tokens=%lld times q_heads=%lld passes 2^28", p->tokens, p->q_heads);
    if (p->batch < 0 || p->batch > kMaxBatch) return fail_in(fn, BG_ERR_SHAPE, "batch=%lld out of range", p->batch);
    if (p->q_heads < a->c.heads || p->q_heads > 16384 || p->q_heads % a->c.heads)
        return fail_in(fn, BG_ERR_SHAPE, "q_heads=%lld is not a multiple of kv_heads=%lld", p->q_heads, a->c.heads);
    if (p->max_pages < 1 || p->max_pages > INT32_MAX) return fail_in(fn, BG_ERR_SHAPE, "max_pages=%lld out of range", p->max_pages);
    // positions less a window and a call's queries have to fit 32 bits
    if (p->max_pages > ((INT32_MAX - 2 * kMaxTokens) >> a->c.page_shift))
        return fail_in(fn, BG_ERR_SHAPE, "max_pages=%lld pages of %lld tokens pass 2^31 - 2^25 positions", p->max_pages, p->cache->page_size);
    if (p->max_q < 1 || p->max_q > kMaxTokens) return fail_in(fn, BG_ERR_SHAPE, "max_q=%lld out of range", p->max_q);
    if (p->max_kv < 0) return fail_in(fn, BG_ERR_SHAPE, "max_kv=%lld is negative", p->max_kv);
    if (p->window < 0 || p->sinks < 0) return fail_in(fn, BG_ERR_SHAPE, "window=%lld and sinks=%lld must not be negative", p->window, p->sinks);
    if (p->q_token_stride % 8 || p->q_head_stride % 8)
        return fail_in(fn, BG_ERR_ALIGN, "q strides %lld and %lld must be multiples of 8 elements", p->q_token_stride, p->q_head_stride);
    if (!(p->scale > 0.0f) || p->scale > 3.0e38f) return fail_in(fn, BG_ERR_SHAPE, "scale must be positive and finite");
    if (!p->cu_q && (p->tokens != p->batch || p->max_q != 1))
        return fail_in(fn, BG_ERR_SHAPE, "without cu_q every sequence has one query: tokens=%lld, batch=%lld", p->tokens, p->batch);
    if (tree && (p->tree_words < 1 || p->tree_words > 1024))
        return fail_in(fn, BG_ERR_SHAPE, "tree_words=%lld out of range", p->tree_words);
    if (tree && p->window) return fail_in(fn, BG_ERR_UNSUPPORTED, "a window of %lld with a tree", p->window);
    if (pointers && p->tokens > 0 && p->batch > 0) {
        if (!p->q || !p->out || !p->block_table || !p->kv_lens || (tree && !p->tree))
            return fail_in(fn, BG_ERR_NULL, "q, out, block_table, kv_lens (and tree) must be non-NULL");
        if (!aligned16(p->q) || !aligned16(p->out)) return fail_in(fn, BG_ERR_ALIGN, "q and out must be 16-byte aligned");
        if ((reinterpret_cast<uintptr_t>(p->block_table) | reinterpret_cast<uintptr_t>(p->kv_lens) |
             reinterpret_cast<uintptr_t>(p->cu_q) | reinterpret_cast<uintptr_t>(p->lse)) & 3u)
            return fail_in(fn, BG_ERR_ALIGN, "block_table, kv_lens, cu_q and lse must be 4-byte aligned");
        if (tree && (reinterpret_cast<uintptr_t>(p->tree) & 7u)) return fail_in(fn, BG_ERR_ALIGN, "tree must be 8-byte aligned");
    }
    a->q = p->q;
    a->q_ts = p->q_token_stride;
    a->q_hs = p->q_head_stride;
    a->bf16 = p->dtype == BG_BF16;
    a->tokens = p->tokens;
    a->q_heads = p->q_heads;
    a->table = p->block_table;
    a->max_pages = p->max_pages;
    a->kv_lens = p->kv_lens;
    a->cu_q = p->cu_q;
    a->batch = p->batch;
    a->max_q = p->max_q < p->tokens ? p->max_q : p->tokens;
    const int64_t room = p->max_pages << a->c.page_shift;
    a->max_kv = p->max_kv == 0 || p->max_kv > room ? room : p->max_kv;
    a->window = p->window >= room ? 0 : p->window;      // such a window holds every position
    a->sinks = a->window ? (p->sinks > INT32_MAX ? INT32_MAX : p->sinks) : 0;
    a->tree = tree ? p->tree : nullptr;
    a->tree_words = tree ? p->tree_words : 0;
    a->scale = p->scale;
    a->out = p->out;
    a->lse = p->lse;
    return BG_OK;
}

// What `sc` asks of the scores, checked.
bg_status kv_scores(const char* fn, const bg_kv_scores* sc, bool tree, bg::KvAttnArgs* a) {
    if (!(sc->softcap >= 0.0f) || sc->softcap > 1.0e30f || (sc->softcap > 0.0f && sc->softcap < 1.0e-30f))
        return fail_in(fn, BG_ERR_SHAPE, "softcap must be 0 or lie in 1e-30 .. 1e30");
    if (tree && (sc->slopes || sc->prefix_lens)) return fail_in(fn, BG_ERR_UNSUPPORTED, "slopes or prefix_lens with a tree");
    if (!aligned(sc->slopes, 4) || !aligned(sc->prefix_lens, 4)) return fail_in(fn, BG_ERR_ALIGN, "slopes and prefix_lens must be 4-byte aligned");
    const bool caps = sc->softcap > 0.0f;
    a->cap = caps ? (float)(sc->softcap * 0x1.71547652b82fep0) : 1.0f;
    a->cap_inv = caps ? (float)(1.0 / (sc->softcap * 0x1.71547652b82fep0)) : 0.0f;
    a->slopes = sc->slopes;
    a->prefix = sc->prefix_lens;
    a->scored = caps || a->slopes || a->prefix;
    return BG_OK;
}

bg_status kv_attn_impl(const char* fn, const bg_kv_attn* p, bool tree, const bg_kv_scores* sc, void* ws, int64_t ws_bytes, void* stream) {
    bg::KvAttnArgs a{};
    bg_status st = kv_attn_args(fn, p, tree, true, &a);
    if (st == BG_OK && sc) st = kv_scores(fn, sc, tree, &a);
    if (st != BG_OK) return st;
    if (a.tokens == 0 || a.batch == 0) {
        g_last_error[0] = '\0';
        return BG_OK;
    }
    const int64_t need = bg::kv_attn_workspace(a);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail_in(fn, BG_ERR_WORKSPACE, "workspace of %lld bytes needed (got %lld)", need, ws ? ws_bytes : 0);
    if (ws && !aligned16(ws)) return fail_in(fn, BG_ERR_ALIGN, "the workspace must be 16-byte aligned");
    note_kernel(bg::launch_kv_attn(a, ws, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

}  // namespace

BG_EXPORT bg_status kv_cache_write(const bg_kv_cache* cache, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                                   const void* v, int64_t v_token_stride, int64_t v_head_stride, int x_dtype,
                                   const int64_t* slots, int64_t tokens, void* stream) {
    const char* fn = "kv_cache_write";
    bg::KvCache c;
    const bg_status st = kv_cache_of(fn, cache, &c);
    if (st != BG_OK) return st;
    if (x_dtype != BG_F32 && x_dtype != BG_F16 && x_dtype != BG_BF16)
        return fail_in(fn, BG_ERR_DTYPE, "x_dtype %lld is not F32/F16/BF16", x_dtype);
    if (tokens < 0 || tokens > kMaxTokens) return fail_in(fn, BG_ERR_SHAPE, "tokens=%lld out of range", tokens);
    if (tokens == 0) {
        g_last_error[0] = '\0';
        return BG_OK;
    }
    if (!k || !v || !slots) return fail_in(fn, BG_ERR_NULL, "k, v and slots must be non-NULL");
    const int64_t unit = x_dtype == BG_F32 ? 4 : 8;   // elements in 16 bytes
    if (k_token_stride % unit || k_head_stride % unit || v_token_stride % unit || v_head_stride % unit)
        return fail_in(fn, BG_ERR_ALIGN, "strides must be multiples of 16 bytes (%lld elements)", unit);
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 7u))
        return fail_in(fn, BG_ERR_ALIGN, "k and v must be 16-byte aligned, slots 8-byte aligned");
    const bg::KvRows x{k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    note_kernel(bg::launch_kv_write(c, x, x_dtype, tokens, slots, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

BG_EXPORT bg_status kv_cache_read(const bg_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                                  int out_dtype, void* stream) {
    const char* fn = "kv_cache_read";
    bg::KvCache c;
    const bg_status st = kv_cache_of(fn, cache, &c);
    if (st != BG_OK) return st;
    if (out_dtype != BG_F32 && out_dtype != BG_F16 && out_dtype != BG_BF16)
        return fail_in(fn, BG_ERR_DTYPE, "out_dtype %lld is not F32/F16/BF16", out_dtype);
    if (tokens < 0 || tokens > kMaxTokens) return fail_in(fn, BG_ERR_SHAPE, "tokens=%lld out of range", tokens);
    if (tokens == 0) {
        g_last_error[0] = '\0';
        return BG_OK;
    }
    if (!k || !v || !slots) return fail_in(fn, BG_ERR_NULL, "k, v and slots must be non-NULL");
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 7u))
        return fail_in(fn, BG_ERR_ALIGN, "k and v must be 16-byte aligned, slots 8-byte aligned");
    note_kernel(bg::launch_kv_read(c, slots, tokens, out_dtype, k, v, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

BG_EXPORT bg_status kv_attn(const bg_kv_attn* args, void* workspace, int64_t workspace_bytes, void* stream) {
    return kv_attn_impl("kv_attn", args, false, nullptr, workspace, workspace_bytes, stream);
}

BG_EXPORT bg_status kv_attn_tree(const bg_kv_attn* args, void* workspace, int64_t workspace_bytes, void* stream) {
    return kv_attn_impl("kv_attn_tree", args, true, nullptr, workspace, workspace_bytes, stream);
}

BG_EXPORT bg_status kv_attn_scored(const bg_kv_attn* args, const bg_kv_scores* scores, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "kv_attn_scored";
    if (!scores) return fail_in(fn, BG_ERR_NULL, "scores must be non-NULL");
    return kv_attn_impl(fn, args, args && args->tree_words > 0, scores, workspace, workspace_bytes, stream);
}

BG_EXPORT int64_t kv_attn_workspace_bytes(const bg_kv_attn* args) {
    bg::KvAttnArgs a{};
    if (kv_attn_args("kv_attn_workspace_bytes", args, args && args->tree_words > 0, false, &a) != BG_OK) return 0;
    if (a.tokens == 0 || a.batch == 0) return 0;
    return bg::kv_attn_workspace(a);
}

namespace {

constexpr int64_t kMaxPoolPages = int64_t(1) << 30;

bg::Span ints(const void* p, int64_t n) { return bg::Span(p, 4 * (uint64_t)n); }

// The pool of `fn`, checked.
bg_status kv_pool_of(const char* fn, const bg_kv_pool* p, bg::KvPool* out) {
    if (!p) return fail_in(fn, BG_ERR_NULL, "pool must be non-NULL");
    if (!p->block_table || !p->lens || !p->free_pages || !p->state || (p->window && !p->gone))
        return fail_in(fn, BG_ERR_NULL, "the pool's arrays must be non-NULL");
    if (p->batch < 1 || p->batch > kMaxBatch) return fail_in(fn, BG_ERR_SHAPE, "batch=%lld out of range", p->batch);
    if (p->page_size < 16 || p->page_size > 1024 || (p->page_size & (p->page_size - 1)))
        return fail_in(fn, BG_ERR_SHAPE, "page_size %lld is not a power of two in 16..1024", p->page_size);
    if (p->pages < 1 || p->pages > kMaxPoolPages) return fail_in(fn, BG_ERR_SHAPE, "pages=%lld out of range", p->pages);
    const int shift = __builtin_ctz((unsigned)p->page_size);
    if (p->max_pages < 1 || p->max_pages > ((INT32_MAX - 2 * kMaxTokens) >> shift))
        return fail_in(fn, BG_ERR_SHAPE, "max_pages=%lld pages of %lld tokens are none, or pass 2^31 - 2^25 positions", p->max_pages, p->page_size);
    if (p->window < 0 || p->sinks < 0) return fail_in(fn, BG_ERR_SHAPE, "window=%lld and sinks=%lld must not be negative", p->window, p->sinks);
    if (!aligned(p->block_table, 4) || !aligned(p->lens, 4) || !aligned(p->gone, 4) || !aligned(p->free_pages, 4) || !aligned(p->state, 4))
        return fail_in(fn, BG_ERR_ALIGN, "the pool's arrays must be 4-byte aligned");
    auto clamped = [](int64_t n) { return (int)(n > INT32_MAX ? INT32_MAX : n); };
    *out = bg::KvPool{p->block_table, p->lens, p->gone, p->free_pages, p->state, p->batch, p->max_pages, p->pages,
                      shift, clamped(p->window), clamped(p->sinks)};
    return BG_OK;
}

// The rows of `fn`, checked; kv_heads and dim: the cache's, or the arguments' own (0).
bg_status rope_args(const char* fn, const bg_qk_rope* p, const bg::KvCache* cache, bg::RopeArgs* a, int* dim) {
    if (!p) return fail_in(fn, BG_ERR_NULL, "args must be non-NULL");
    const int kv_heads = cache ? cache->heads : p->kv_heads;
    *dim = cache ? cache->dim : p->head_dim;
    if (p->x_dtype != BG_F32 && p->x_dtype != BG_F16 && p->x_dtype != BG_BF16)
        return fail_in(fn, BG_ERR_DTYPE, "x_dtype %lld is not F32/F16/BF16", p->x_dtype);
    if ((p->q_weight || p->k_weight) && p->weight_dtype != p->x_dtype && p->weight_dtype != BG_F32)
        return fail_in(fn, BG_ERR_DTYPE, "weight_dtype %lld is neither x_dtype nor F32", p->weight_dtype);
    if (*dim != 64 && *dim != 128 && *dim != 256) return fail_in(fn, BG_ERR_SHAPE, "head_dim %lld is not 64, 128 or 256", *dim);
    if (p->rot < 0 || p->rot > *dim || p->rot % 8)
        return fail_in(fn, BG_ERR_SHAPE, "rot=%lld is not a multiple of 8 up to head_dim=%lld", p->rot, *dim);
    if (p->q_heads < 0 || p->q_heads > 16384 || kv_heads < 0 || kv_heads > 16384 || p->q_heads + kv_heads == 0)
        return fail_in(fn, BG_ERR_SHAPE, "q_heads=%lld, kv_heads=%lld out of range", p->q_heads, kv_heads);
    if (p->tokens < 0 || p->tokens > kMaxTokens) return fail_in(fn, BG_ERR_SHAPE, "tokens=%lld out of range", p->tokens);
    const int64_t heads = p->q_heads > kv_heads ? p->q_heads : kv_heads;
    if (p->tokens * heads > (int64_t(1) << 28)) return fail_in(fn, BG_ERR_SHAPE, "tokens=%lld times %lld heads pass 2^28", p->tokens, heads);
    if (!(p->eps >= 0.0) || p->eps > 1.0e30 || !(p->weight_offset >= -1.0e30 && p->weight_offset <= 1.0e30))
        return fail_in(fn, BG_ERR_SHAPE, "eps must be at least 0, eps and weight_offset finite");
    const int64_t unit = p->x_dtype == BG_F32 ? 4 : 8;   // elements in 16 bytes
    const bool q = p->q_heads > 0, k = kv_heads > 0, k_out = k && !cache;
    if ((q && (p->q_token_stride % unit || p->q_head_stride % unit || p->q_out_token_stride % unit || p->q_out_head_stride % unit)) ||
        (k && (p->k_token_stride % unit || p->k_head_stride % unit)) || (k_out && (p->k_out_token_stride % unit || p->k_out_head_stride % unit)) ||
        (cache && (p->v_token_stride % unit || p->v_head_stride % unit)))
        return fail_in(fn, BG_ERR_ALIGN, "strides must be multiples of 16 bytes (%lld elements)", unit);
    if (p->tokens > 0) {
        if ((q && (!p->q || !p->q_out)) || (k && !p->k) || (k_out && !p->k_out) || (cache && (!p->v || !p->slots)))
            return fail_in(fn, BG_ERR_NULL, "the rows of queries and keys, their outputs, v and slots must be non-NULL");
        if (p->rot && (!p->positions || !p->freqs)) return fail_in(fn, BG_ERR_NULL, "positions and freqs must be non-NULL");
        if ((q && (!aligned16(p->q) || !aligned16(p->q_out))) || (k && !aligned16(p->k)) || (k_out && !aligned16(p->k_out)) ||
            (cache && !aligned16(p->v)) || !aligned16(p->q_weight) || !aligned16(p->k_weight))
            return fail_in(fn, BG_ERR_ALIGN, "rows and weights must be 16-byte aligned");
        if ((p->rot && (!aligned(p->positions, 4) || !aligned(p->freqs, 8))) || (cache && !aligned(p->slots, 8)))
            return fail_in(fn, BG_ERR_ALIGN, "positions must be 4-byte aligned, freqs and slots 8-byte aligned");
        // a block writes its rows while others have theirs yet to read
        const int64_t size = 16 / unit;
        auto rows = [&](const void* at, int64_t ts, int64_t hs, int n) { return bg::RowSet(at, p->tokens, ts * size, n, hs * size, *dim * size); };
        const bg::RowSet in[3] = {rows(p->q, p->q_token_stride, p->q_head_stride, p->q_heads), rows(p->k, p->k_token_stride, p->k_head_stride, kv_heads),
                                  rows(p->v, p->v_token_stride, p->v_head_stride, kv_heads)};
        const bg::RowSet out[2] = {rows(p->q_out, p->q_out_token_stride, p->q_out_head_stride, p->q_heads),
                                   rows(p->k_out, p->k_out_token_stride, p->k_out_head_stride, kv_heads)};
        const bool given[3] = {q, k, cache != nullptr}, written[2] = {q, k_out};
        for (int o = 0; o < 2; ++o) {
            if (!written[o]) continue;
            if (!out[o].distinct()) return fail_in(fn, BG_ERR_UNSUPPORTED, o == 0 ? "q_out's rows overlap" : "k_out's rows overlap");
            for (int i = 0; i < 3; ++i)
                if (given[i] && !(i == o && out[o].same(in[i])) && !bg::apart(out[o], in[i]))
                    return fail_in(fn, BG_ERR_UNSUPPORTED, o == 0 ? "q_out overlaps q (other than as a whole), k or v" : "k_out overlaps k (other than as a whole) or q");
        }
        if (written[0] && written[1] && !bg::apart(out[0], out[1])) return fail_in(fn, BG_ERR_UNSUPPORTED, "q_out and k_out overlap");
    }
    *a = bg::RopeArgs{p->q, p->k, p->v, p->q_out, p->k_out, p->q_token_stride, p->q_head_stride, p->k_token_stride, p->k_head_stride,
                      p->v_token_stride, p->v_head_stride, p->q_out_token_stride, p->q_out_head_stride, p->k_out_token_stride,
                      p->k_out_head_stride, p->q_weight, p->k_weight, p->positions, p->freqs, p->slots, p->tokens, p->q_heads, kv_heads,
                      p->rot, p->interleaved != 0, p->weight_dtype == BG_F32, p->eps, p->weight_offset};
    return BG_OK;
}

bg_status rope_impl(const char* fn, const bg_qk_rope* args, const bg::KvCache* cache, void* stream) {
    bg::RopeArgs a;
    int dim = 0;
    const bg_status st = rope_args(fn, args, cache, &a, &dim);
    if (st != BG_OK) return st;
    if (a.tokens == 0) {
        g_last_error[0] = '\0';
        return BG_OK;
    }
    note_kernel(bg::launch_qk_rope(a, args->x_dtype, dim, cache, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

}  // namespace

BG_EXPORT bg_status kv_plan(const bg_kv_pool* pool, const int32_t* q_lens, int64_t tokens, int advance, int32_t* cu_q,
                            int32_t* kv_lens, int32_t* served, int32_t* positions, int64_t* slots, void* stream) {
    const char* fn = "kv_plan";
    bg::KvPool p;
    const bg_status st = kv_pool_of(fn, pool, &p);
    if (st != BG_OK) return st;
    if (tokens < 0 || tokens > kMaxTokens) return fail_in(fn, BG_ERR_SHAPE, "tokens=%lld out of range", tokens);
    if (!q_lens || !cu_q || !kv_lens || !served || (tokens > 0 && (!positions || !slots)))
        return fail_in(fn, BG_ERR_NULL, "q_lens, cu_q, kv_lens, served, positions and slots must be non-NULL");
    if (!aligned(q_lens, 4) || !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(served, 4) || !aligned(positions, 4) || !aligned(slots, 8))
        return fail_in(fn, BG_ERR_ALIGN, "lengths, offsets and positions must be 4-byte aligned, slots 8-byte aligned");
    // the first block writes these while others read
    const bg::Span asked = ints(q_lens, p.batch), out[] = {ints(cu_q, p.batch + 1), ints(kv_lens, p.batch), ints(served, p.batch), ints(positions, tokens),
                                                           ints(slots, 2 * tokens)};
    const bg::Span held[] = {ints(p.table, p.batch * p.max_pages), ints(p.free, p.pages), ints(p.state, 2), ints(p.lens, p.batch),
                             ints(p.gone, p.gone ? p.batch : 0)};
    for (const bg::Span& x : out) {
        for (const bg::Span& y : out)
            if (&x != &y && !bg::apart(x, y)) return fail_in(fn, BG_ERR_UNSUPPORTED, "two outputs overlap");
        for (const bg::Span& y : held)
            if (!bg::apart(x, y)) return fail_in(fn, BG_ERR_UNSUPPORTED, "an output overlaps the pool");
        if (!bg::apart(x, asked)) return fail_in(fn, BG_ERR_UNSUPPORTED, "q_lens overlaps an output");
    }
    for (int i = 0; i < 4; ++i)
        if (!bg::apart(asked, held[i]) && !(i == 3 && q_lens == p.lens)) return fail_in(fn, BG_ERR_UNSUPPORTED, "q_lens overlaps what the step writes of the pool");
    const bg::KvPlan o{q_lens, tokens, advance != 0, cu_q, kv_lens, served, positions, slots};
    note_kernel(bg::launch_kv_plan(p, o, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

BG_EXPORT bg_status kv_release(const bg_kv_pool* pool, const int32_t* keep, void* stream) {
    const char* fn = "kv_release";
    bg::KvPool p;
    const bg_status st = kv_pool_of(fn, pool, &p);
    if (st != BG_OK) return st;
    if (!aligned(keep, 4)) return fail_in(fn, BG_ERR_ALIGN, "keep must be 4-byte aligned");
    if (keep && keep != p.lens && keep != p.gone)           // these are read as they are written, a sequence by one thread
        for (const bg::Span& y : {ints(p.table, p.batch * p.max_pages), ints(p.free, p.pages), ints(p.state, 2), ints(p.lens, p.batch),
                                  ints(p.gone, p.gone ? p.batch : 0)})
            if (!bg::apart(ints(keep, p.batch), y)) return fail_in(fn, BG_ERR_UNSUPPORTED, "keep overlaps the pool");
    note_kernel(bg::launch_kv_release(p, keep, static_cast<hipStream_t>(stream)));
    return launched(fn);
}

BG_EXPORT bg_status qk_norm_rope(const bg_qk_rope* args, void* stream) { return rope_impl("qk_norm_rope", args, nullptr, stream); }

BG_EXPORT bg_status kv_cache_write_rope(const bg_kv_cache* cache, const bg_qk_rope* args, void* stream) {
    const char* fn = "kv_cache_write_rope";
    bg::KvCache c;
    const bg_status st = kv_cache_of(fn, cache, &c);
    return st == BG_OK ? rope_impl(fn, args, &c, stream) : st;
}

BG_EXPORT const char* bg_status_string(int status) {
    switch (status) {
        case BG_OK: return "ok";
        case BG_ERR_NULL: return "null pointer";
        case BG_ERR_SHAPE: return "unsupported shape";
        case BG_ERR_ALIGN: return "misaligned pointer";
        case BG_ERR_DTYPE: return "unsupported dtype";
        case BG_ERR_UNSUPPORTED: return "unsupported combination";
        case BG_ERR_HIP: return "HIP runtime error";
        case BG_ERR_WORKSPACE: return "workspace missing or too small";
        default: return "unknown status";
    }
}

BG_EXPORT const char* bg_last_error(void) { return g_last_error; }

BG_EXPORT int bg_pack_format_version(void) { return BG_PACK_FORMAT_VERSION; }

BG_EXPORT const char* bg_last_kernel(void) { return g_last_kernel; }
