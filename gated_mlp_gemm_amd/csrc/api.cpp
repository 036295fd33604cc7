// C ABI of the fused SwiGLU GEMM library: argument validation, the M-based
// dispatcher between the two fused variants, and kernel launches.
//
// Every argument is checked before the first HIP call, so an invalid call
// launches nothing (and can be exercised on a machine without a GPU).
#include "swiglu.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cmath>
#include <cstring>
#include <atomic>
#include <chrono>
#include <mutex>

#include "arrivals.hpp"
#include "launch.hpp"

namespace {

thread_local char g_last_error[512] = "";

int fail(int status, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return status;
}

int ok() {
    g_last_error[0] = '\0';
    return SWIGLU_OK;
}

constexpr int64_t kMaxM = 2147483647;     // 2^31 - 1
constexpr int64_t kMaxK = int64_t(1) << 21;
constexpr int64_t kMaxN = int64_t(1) << 22;
// Built-in M threshold of the dispatcher: every M.  On MI355X variant I was
// faster than variant S at 44 of 45 measured (M, K, N) points -- M from 128 to
// 16384 on each of the five K x N shapes of the workloads, by 10-20 % at large
// M -- and within 1-8 % (run to run) at the other (M = 128, K = 1536, N =
// 8960), so AUTO runs I unless SWIGLU_M_SWITCH sets a smaller threshold.
constexpr int64_t kDefaultMSwitch = kMaxM;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

int check_gemm_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0) return fail(SWIGLU_ERR_SHAPE, "negative size M=%lld N=%lld", (long long)M, (long long)N);
    if (K < 8) return fail(SWIGLU_ERR_SHAPE, "K=%lld must be >= 8", (long long)K);
    if (K % 8 != 0 || N % 8 != 0)
        return fail(SWIGLU_ERR_SHAPE, "K=%lld and N=%lld must be multiples of 8", (long long)K, (long long)N);
    if (M > kMaxM || K > kMaxK || N > kMaxN)
        return fail(SWIGLU_ERR_SHAPE, "size beyond limits (M<=2^31-1, K<=2^21, N<=2^22)");
    if (swiglu::max_tiles(M, 2 * N) > 2147483647)
        return fail(SWIGLU_ERR_SHAPE, "tile grid too large");
    return SWIGLU_OK;
}

// The down projection Out [M][D] = H [M][N] . W3 reduces over N: N is its
// K-like dimension (multiple of 8, at most 2^21) and D its column count.
int check_down_shape(int64_t M, int64_t N, int64_t D) {
    if (M < 0 || D < 0) return fail(SWIGLU_ERR_SHAPE, "negative size M=%lld D=%lld", (long long)M, (long long)D);
    if (N < 8) return fail(SWIGLU_ERR_SHAPE, "N=%lld must be >= 8", (long long)N);
    if (N % 8 != 0 || D % 8 != 0)
        return fail(SWIGLU_ERR_SHAPE, "N=%lld and D=%lld must be multiples of 8", (long long)N, (long long)D);
    if (M > kMaxM || N > kMaxK || D > kMaxN)
        return fail(SWIGLU_ERR_SHAPE, "size beyond limits (M<=2^31-1, N<=2^21, D<=2^22)");
    if (swiglu::max_tiles(M, D) > 2147483647) return fail(SWIGLU_ERR_SHAPE, "tile grid too large");
    return SWIGLU_OK;
}

// swiglu_describe_launch's codes for the down projection of the gated MLP
// and for the FP8 fused call.
constexpr int kDescribeDownProj = -2;
constexpr int kDescribeFp8 = -3;

// Per-device cache: state 1 = gfx950, -1 = other architecture, 0 = not yet
// queried; and the device's compute-unit count (sizes the split-tail schedule).
std::mutex g_dev_mutex;
int g_dev_state[256];
int g_dev_cus[256];


int check_device(int *cus = nullptr) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(SWIGLU_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= 256) return fail(SWIGLU_ERR_UNSUPPORTED, "device ordinal %d", dev);
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (g_dev_state[dev] == 0) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess)
            return fail(SWIGLU_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
        g_dev_state[dev] = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
        g_dev_cus[dev] = prop.multiProcessorCount;
    }
    if (g_dev_state[dev] != 1)
        return fail(SWIGLU_ERR_UNSUPPORTED, "device %d is not gfx950 (MI355X)", dev);
    if (cus) *cus = g_dev_cus[dev];
    return SWIGLU_OK;
}

// SWIGLU_I_TILE=256 or 128 forces the tile of variant I and the ablation
// GEMMs above M = 128, and variant I's 128x64 (256) or 128x128 (128) tiles at
// M <= 128 (testing, measurement); anything else: the cost model / rule.
int tile_override() {
    const char *s = std::getenv("SWIGLU_I_TILE");
    if (s == nullptr) return 0;
    if (std::strcmp(s, "256") == 0) return 256;
    if (std::strcmp(s, "128") == 0) return 128;
    return 0;
}

// SWIGLU_TAIL=whole, split or quarter forces how the tiles of a partly idle
// last round run (split only takes effect with a workspace; quarter only for
// the 256x256 tile); fixup forces variant I at M <= 128 to split all its
// tiles along K and reduce them in the kernel (with a workspace; whole keeps
// it from doing so); unset or anything else: the cost model decides.
int tail_override() {
    const char *s = std::getenv("SWIGLU_TAIL");
    if (s == nullptr) return swiglu::kTailAuto;
    if (std::strcmp(s, "whole") == 0) return swiglu::kTailWhole;
    if (std::strcmp(s, "split") == 0) return swiglu::kTailPieces;
    if (std::strcmp(s, "quarter") == 0) return swiglu::kTailQuarters;
    if (std::strcmp(s, "fixup") == 0) return swiglu::kTailFixup;
    return swiglu::kTailAuto;
}

// The tag of a launch whose workgroups meet (arrivals.hpp): a number of its upper 52
// bits that no other launch of this process has, spread over all of them (the step is odd),
// from a start that other processes hardly share.
uint64_t next_arrival_tag() {
    static std::atomic<uint64_t> next{
        static_cast<uint64_t>(std::chrono::system_clock::now().time_since_epoch().count()) ^
        (static_cast<uint64_t>(reinterpret_cast<uintptr_t>(&g_dev_mutex)) << 20)};
    return next.fetch_add(0x9E3779B97F4A7C15u, std::memory_order_relaxed) << swiglu::kArrivalBits;
}

swiglu::GemmWorkspace make_ws(void *workspace, uint64_t bytes, int cus) {
    swiglu::GemmWorkspace ws{};
    ws.base = bytes > 0 ? workspace : nullptr;
    ws.bytes = workspace ? bytes : 0;
    ws.cus = cus;
    ws.tile = tile_override();
    ws.tail = tail_override();
    ws.tag = next_arrival_tag();
    return ws;
}

// Library-owned scratch of swiglu_fused_gemm_noalloc: the split-tail partials
// of one call (one fp32 256 x 256 slot per compute unit of a 256-CU device).
// A file-scope device array, so the library allocates nothing at call time;
// each device the library runs on holds its own copy until the process ends.
// Host code never uses the array's name as an address: the per-device device
// address comes from hipGetSymbolAddress (scratch_on_device).
constexpr uint64_t kScratchBytes = uint64_t(64) << 20;
static __device__ __align__(256) unsigned char scratch[kScratchBytes];
void *g_scratch_ptr[256];   // per device, guarded by g_dev_mutex

// Device address of this device's `scratch`, looked up once per device with
// that device current (the caller's current device).
int scratch_on_device(void **ptr) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(SWIGLU_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= 256) return fail(SWIGLU_ERR_UNSUPPORTED, "device ordinal %d", dev);
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (g_scratch_ptr[dev] == nullptr) {
        void *p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || p == nullptr)
            return fail(SWIGLU_ERR_HIP, "hipGetSymbolAddress(scratch): %s", hipGetErrorString(e));
        g_scratch_ptr[dev] = p;
    }
    *ptr = g_scratch_ptr[dev];
    return SWIGLU_OK;
}

int check_workspace(const void *workspace, uint64_t bytes) {
    if (workspace && bytes > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(SWIGLU_ERR_ALIGN, "workspace must be 256-byte aligned");
    return SWIGLU_OK;
}

// The operands of a call, for the checks that every pointer is there, is
// aligned, and that no output overlaps another operand.
struct Operand {
    const char *name;
    const void *p;
    int64_t bytes;
    uint32_t align;     // bytes, a power of two
    bool output;
    bool optional;      // may be NULL
};
int check_operands(const Operand *ops, int n) {
    for (int i = 0; i < n; ++i)
        if (!ops[i].p && !ops[i].optional) return fail(SWIGLU_ERR_NULL, "%s is required", ops[i].name);
    for (int i = 0; i < n; ++i)
        if (reinterpret_cast<uintptr_t>(ops[i].p) & (ops[i].align - 1))
            return fail(SWIGLU_ERR_ALIGN, "%s must be %u-byte aligned", ops[i].name, ops[i].align);
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && ops[i].output && ops[i].p && ops[j].p &&
                overlap(ops[i].p, ops[i].bytes, ops[j].p, ops[j].bytes))
                return fail(SWIGLU_ERR_ALIAS, "%s overlaps %s", ops[i].name, ops[j].name);
    return SWIGLU_OK;
}

int check_route(int logits_type, int64_t M, int64_t E, int64_t k) {
    if (logits_type != SWIGLU_F32 && logits_type != SWIGLU_BF16)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown logits type %d", logits_type);
    if (M < 0 || M > kMaxM) return fail(SWIGLU_ERR_SHAPE, "M=%lld outside [0, 2^31 - 1]", (long long)M);
    if (E < 1 || E > swiglu::kMaxRouteE)
        return fail(SWIGLU_ERR_SHAPE, "E=%lld outside [1, %d]", (long long)E, swiglu::kMaxRouteE);
    if (k < 1 || k > E || k > swiglu::kMaxRouteK)
        return fail(SWIGLU_ERR_SHAPE, "k=%lld outside [1, min(E, %d)]", (long long)k,
                    swiglu::kMaxRouteK);
    return SWIGLU_OK;
}

int check_lora(int64_t slots, int64_t count, int64_t rank) {
    if (slots < 1 || slots > swiglu::kMaxLoraSlots)
        return fail(SWIGLU_ERR_SHAPE, "slots=%lld outside [1, %d]", (long long)slots,
                    swiglu::kMaxLoraSlots);
    if (rank < 8 || rank > swiglu::kMaxLoraRank || rank % 8 != 0)
        return fail(SWIGLU_ERR_SHAPE, "rank=%lld must be a multiple of 8 in [8, %d]",
                    (long long)rank, swiglu::kMaxLoraRank);
    if (count < 1 || count > swiglu::kMaxLoraCount)
        return fail(SWIGLU_ERR_SHAPE, "count=%lld adapters outside [1, %d]", (long long)count,
                    swiglu::kMaxLoraCount);
    return SWIGLU_OK;
}

// Bytes of the workspace that hold T [M][slots][width], and with the plans of
// the expansion behind it; multiples of 256.
uint64_t lora_t_bytes(int64_t M, int64_t slots, int64_t width) {
    return (static_cast<uint64_t>(M) * slots * width * 4 + 255) & ~uint64_t{255};
}
uint64_t lora_state_bytes(int64_t M, int64_t slots, int64_t width, int64_t count) {
    const uint64_t plans =
        static_cast<uint64_t>((M + 255) / 256) * swiglu::lora_plan_bytes((int)count, (int)slots);
    return lora_t_bytes(M, slots, width) + ((plans + 255) & ~uint64_t{255});
}
int check_lora_workspace(const void *workspace, uint64_t bytes, uint64_t need) {
    if (!workspace) return fail(SWIGLU_ERR_NULL, "workspace is required");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(SWIGLU_ERR_ALIGN, "workspace must be 256-byte aligned");
    if (bytes < need)
        return fail(SWIGLU_ERR_SHAPE, "workspace of %llu bytes, at least %llu are needed",
                    (unsigned long long)bytes, (unsigned long long)need);
    return SWIGLU_OK;
}

// One projection with adapters: the shrink, then the product with the expansion.
hipError_t lora_projection(const uint16_t *X, const uint16_t *W, uint16_t *Y, int64_t M,
                           int64_t cols, int64_t K, bool gated, const swiglu::LoraTable &t,
                           const int32_t *ids, const float *weights, int64_t slots,
                           void *workspace, uint64_t bytes, int cus, hipStream_t s) {
    const int parts = gated ? 2 : 1;
    const uint64_t state = lora_state_bytes(M, slots, parts * t.rank, t.count);
    uint16_t *T = static_cast<uint16_t *>(workspace);
    char *plans = static_cast<char *>(workspace) + lora_t_bytes(M, slots, parts * t.rank);
    // the two launches run in stream order: they share scratch
    swiglu::GemmWorkspace ws = make_ws(static_cast<char *>(workspace) + state, bytes - state, cus);
    const hipError_t e = swiglu::launch_lora_shrink(X, t, ids, weights, (int)slots, T, plans,
                                                    (int)M, (int)K, parts, ws, s);
    if (e != hipSuccess) return e;
    ws.tag = next_arrival_tag();
    return swiglu::launch_lora_project(X, W, Y, (int)M, (int)cols, (int)K, gated, t,
                                       (int)slots, T, plans, ws, s);
}

// Sizes of the training calls: rows of any count are contracted by the weights'
// gradients, and N is also a contraction (2N columns of GU).
constexpr int64_t kMaxTrainM = int64_t(1) << 30;
constexpr int64_t kMaxTrainN = int64_t(1) << 20;
int check_train_shape(int64_t M, int64_t N, int64_t K) {
    int st = check_gemm_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M > kMaxTrainM || N > kMaxTrainN)
        return fail(SWIGLU_ERR_SHAPE, "size beyond limits (M<=2^30, N<=2^20)");
    if (swiglu::max_tiles(2 * N, K) > 2147483647 || swiglu::max_tiles(M, K) > 2147483647)
        return fail(SWIGLU_ERR_SHAPE, "tile grid too large");
    return SWIGLU_OK;
}
int check_down_backward_shape(int64_t M, int64_t N, int64_t D) {
    int st = check_down_shape(M, N, D);
    if (st != SWIGLU_OK) return st;
    if (D < 8) return fail(SWIGLU_ERR_SHAPE, "D=%lld must be >= 8", (long long)D);
    if (M > kMaxTrainM || D > kMaxK || swiglu::max_tiles(M, N) > 2147483647 ||
        swiglu::max_tiles(D, N) > 2147483647)
        return fail(SWIGLU_ERR_SHAPE, "size beyond limits (M<=2^30, D<=2^21, tile grids)");
    return SWIGLU_OK;
}
int check_stage_backward_shape(int64_t M, int64_t N, int64_t K) {
    int st = check_train_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (N < 8) return fail(SWIGLU_ERR_SHAPE, "N=%lld must be >= 8", (long long)N);
    return SWIGLU_OK;
}
int check_block_backward_shape(int64_t M, int64_t N, int64_t K) {
    int st = check_train_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_down_shape(M, N, K);
    return st;
}
int check_grad_type(int grad_type) {
    if (grad_type != SWIGLU_F32 && grad_type != SWIGLU_BF16)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown gradient type %d", grad_type);
    return SWIGLU_OK;
}
// A contraction over 4-bit weights: whole groups.
int check_mx4_groups(const char *name, int64_t n) {
    if (n < 32 || n % 32 != 0)
        return fail(SWIGLU_ERR_SHAPE, "%s=%lld must be a positive multiple of 32", name, (long long)n);
    return SWIGLU_OK;
}
int check_mx4_matrix(int64_t rows, int64_t K) {
    int st = check_mx4_groups("K", K);
    if (st != SWIGLU_OK) return st;
    if (rows < 0 || rows > 2 * kMaxN || K > kMaxK)
        return fail(SWIGLU_ERR_SHAPE, "size beyond limits (0<=rows<=2^23, K<=2^21)");
    return SWIGLU_OK;
}
int grad_size(int grad_type) { return grad_type == SWIGLU_F32 ? 4 : 2; }
// A sum that a weight's gradient is added to may be the gradient itself.
const void *add_operand(const void *add, const void *dW) { return add == dW ? nullptr : add; }

int launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(SWIGLU_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return ok();
}

}  // namespace

extern "C" {

const char *swiglu_status_string(int status) {
    switch (status) {
        case SWIGLU_OK: return "ok";
        case SWIGLU_ERR_NULL: return "null pointer";
        case SWIGLU_ERR_SHAPE: return "invalid shape";
        case SWIGLU_ERR_ALIGN: return "pointer not 16-byte aligned";
        case SWIGLU_ERR_UNSUPPORTED: return "unsupported variant or device";
        case SWIGLU_ERR_HIP: return "HIP error";
        case SWIGLU_ERR_ALIAS: return "output overlaps another operand";
        default: return "unknown status";
    }
}

const char *swiglu_last_error(void) { return g_last_error; }

int64_t swiglu_m_switch(void) {
    const char *s = std::getenv("SWIGLU_M_SWITCH");
    if (s != nullptr && *s != '\0') {
        char *end = nullptr;
        const long long v = std::strtoll(s, &end, 10);
        if (end != s && *end == '\0') return v;
    }
    return kDefaultMSwitch;
}

int swiglu_select_variant(int64_t M, int64_t N, int64_t K) {
    (void)N;
    (void)K;
    if (M < 0) return fail(SWIGLU_ERR_SHAPE, "negative M");
    return M <= swiglu_m_switch() ? SWIGLU_VARIANT_I : SWIGLU_VARIANT_S;
}

int swiglu_pack_weights(const uint16_t *W1, const uint16_t *W2, uint16_t *W_fused, int64_t K,
                        int64_t N, void *stream) {
    if (K < 0 || N < 0) return fail(SWIGLU_ERR_SHAPE, "negative size");
    // both are row lengths of 16-byte-chunked rows: N of W1/W2, K of the packed array
    if (K % 8 != 0 || N % 8 != 0)
        return fail(SWIGLU_ERR_SHAPE, "K=%lld and N=%lld must be multiples of 8", (long long)K,
                    (long long)N);
    if (K > kMaxK || N > kMaxN) return fail(SWIGLU_ERR_SHAPE, "size beyond limits");
    if (K == 0 || N == 0) return ok();
    if (!W1 || !W2 || !W_fused) return fail(SWIGLU_ERR_NULL, "W1, W2 and W_fused are required");
    if (!aligned16(W1) || !aligned16(W2) || !aligned16(W_fused))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    const int64_t wbytes = K * N * 2;
    if (overlap(W_fused, 2 * wbytes, W1, wbytes) || overlap(W_fused, 2 * wbytes, W2, wbytes))
        return fail(SWIGLU_ERR_ALIAS, "W_fused overlaps W1 or W2");
    int st = check_device();
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_pack(W1, W2, W_fused, K, N, (hipStream_t)stream), "pack");
}

int swiglu_workspace_size(int64_t M, int64_t N, int64_t K, int variant, uint64_t *bytes) {
    if (!bytes) return fail(SWIGLU_ERR_NULL, "bytes is required");
    *bytes = 0;
    if (variant < -1 || variant > SWIGLU_VARIANT_I)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown variant %d", variant);
    int st = check_gemm_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0) return ok();
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const int v = variant == SWIGLU_AUTO ? swiglu_select_variant(M, N, K) : variant;
    // variant I and the ablation (-1) run the single-accumulator GEMM
    if (v == SWIGLU_VARIANT_I || v == -1) *bytes = swiglu::workspace_bytes_for(cus);
    return ok();
}

int swiglu_describe_launch(int64_t M, int64_t N, int64_t K, int variant,
                           uint64_t workspace_bytes, char *buf, uint64_t buf_bytes) {
    if (!buf || buf_bytes == 0) return fail(SWIGLU_ERR_NULL, "buf is required");
    buf[0] = '\0';
    if (variant < kDescribeFp8 || variant > SWIGLU_VARIANT_I)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown variant %d", variant);
    int st = variant == kDescribeDownProj ? check_down_shape(M, N, K) : check_gemm_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0) {
        std::snprintf(buf, buf_bytes, "nothing (empty problem)");
        return ok();
    }
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    // only the size of the workspace matters for the plan
    const swiglu::GemmWorkspace ws =
        make_ws(workspace_bytes ? reinterpret_cast<void *>(uintptr_t{256}) : nullptr,
                workspace_bytes, cus);
    const int v = variant == SWIGLU_AUTO ? swiglu_select_variant(M, N, K) : variant;
    if (v == kDescribeFp8) {
        swiglu::describe_gemm_fp8((int)M, (int)(2 * N), (int)K, ws, buf, buf_bytes);
    } else if (v == kDescribeDownProj) {
        swiglu::describe_gemm((int)M, (int)K, (int)N, ws, "StoreEpilogue", buf, buf_bytes);
    } else if (v == SWIGLU_VARIANT_S) {
        swiglu::describe_fused_sequential((int)M, (int)N, (int)K, ws, buf, buf_bytes);
    } else if (v == SWIGLU_VARIANT_I) {
        swiglu::describe_gemm((int)M, (int)(2 * N), (int)K, ws, "PairMulEpilogue", buf, buf_bytes,
                              true);
    } else {
        char g[256];
        swiglu::describe_gemm((int)M, (int)N, (int)K, ws, "StoreEpilogue", g, sizeof g);
        std::snprintf(buf, buf_bytes, "2 x %s + silu_mul_kernel", g);
    }
    return ok();
}

int swiglu_describe_backward(int64_t M, int64_t N, int64_t K, int call, int grad_type, int add,
                             uint64_t workspace_bytes, char *buf, uint64_t buf_bytes) {
    if (!buf || buf_bytes == 0) return fail(SWIGLU_ERR_NULL, "buf is required");
    buf[0] = '\0';
    if (call < SWIGLU_DOWN_PROJ_BACKWARD || call > SWIGLU_GATED_MLP_BACKWARD)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown backward call %d", call);
    int st = check_grad_type(grad_type);
    if (st == SWIGLU_OK)
        st = call == SWIGLU_DOWN_PROJ_BACKWARD    ? check_down_backward_shape(M, N, K)
             : call == SWIGLU_FUSED_GEMM_BACKWARD ? check_stage_backward_shape(M, N, K)
                                                  : check_block_backward_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    // only the size of the workspace matters for the plan
    const swiglu::GemmWorkspace ws =
        make_ws(workspace_bytes ? reinterpret_cast<void *>(uintptr_t{256}) : nullptr,
                workspace_bytes, cus);
    swiglu::describe_backward(static_cast<swiglu::BackwardCall>(call), grad_type == SWIGLU_F32, add != 0,
                              (int)M, (int)N, (int)K, ws, buf, buf_bytes);
    return ok();
}

int swiglu_fused_gemm_strided(const uint16_t *A, int64_t lda, const uint16_t *W_fused,
                              uint16_t *Y, int64_t ldy, int64_t M, int64_t N, int64_t K,
                              int variant, void *workspace, uint64_t workspace_bytes,
                              void *stream) {
    if (variant != SWIGLU_AUTO && variant != SWIGLU_VARIANT_S && variant != SWIGLU_VARIANT_I)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown variant %d", variant);
    int st = check_gemm_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (lda < K || lda % 8 != 0 || lda > kMaxK)
        return fail(SWIGLU_ERR_SHAPE, "lda=%lld must be a multiple of 8 in [K, 2^21]",
                    (long long)lda);
    if (ldy < N || ldy > kMaxN)
        return fail(SWIGLU_ERR_SHAPE, "ldy=%lld must lie in [N, 2^22]", (long long)ldy);
    if (M == 0 || N == 0) return ok();
    const int v = variant == SWIGLU_AUTO ? swiglu_select_variant(M, N, K) : variant;
    if (!A || !W_fused || !Y) return fail(SWIGLU_ERR_NULL, "A, W_fused and Y are required");
    if (!aligned16(A) || !aligned16(W_fused) || !aligned16(Y))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    // the memory spans of the strided views (conservative: rows interleaved
    // with another operand's count as overlapping)
    const int64_t abytes = ((M - 1) * lda + K) * 2, ybytes = ((M - 1) * ldy + N) * 2;
    const int64_t wbytes = 2 * K * N * 2;
    if (overlap(Y, ybytes, A, abytes) || overlap(Y, ybytes, W_fused, wbytes))
        return fail(SWIGLU_ERR_ALIAS, "Y overlaps an input");
    st = check_workspace(workspace, workspace_bytes);
    if (st != SWIGLU_OK) return st;
    if (workspace && workspace_bytes > 0 &&
        (overlap(workspace, (int64_t)workspace_bytes, A, abytes) ||
         overlap(workspace, (int64_t)workspace_bytes, W_fused, wbytes) ||
         overlap(workspace, (int64_t)workspace_bytes, Y, ybytes)))
        return fail(SWIGLU_ERR_ALIAS, "workspace overlaps an operand");
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    if (v == SWIGLU_VARIANT_I)
        return launched(swiglu::launch_fused_interleaved(A, (int)lda, W_fused, Y, (int)ldy,
                                                         (int)M, (int)N, (int)K,
                                                         make_ws(workspace, workspace_bytes, cus),
                                                         s),
                        "fused interleaved");
    return launched(swiglu::launch_fused_sequential(A, (int)lda, W_fused, Y, (int)ldy, (int)M,
                                                    (int)N, (int)K,
                                                    make_ws(workspace, workspace_bytes, cus), s),
                    "fused sequential");
}

int swiglu_fused_gemm(const uint16_t *A, const uint16_t *W_fused, uint16_t *Y, int64_t M,
                      int64_t N, int64_t K, int variant, void *workspace,
                      uint64_t workspace_bytes, void *stream) {
    // contiguous rows: lda = K, ldy = N (validated by the strided entry point
    // after the shape check, so the shape errors are reported first)
    return swiglu_fused_gemm_strided(A, K, W_fused, Y, N, M, N, K, variant, workspace,
                                     workspace_bytes, stream);
}

int swiglu_fused_gemm_noalloc(const uint16_t *A, const uint16_t *W_fused, uint16_t *Y,
                              int64_t M, int64_t N, int64_t K, int variant, void *stream) {
    if (variant != SWIGLU_AUTO && variant != SWIGLU_VARIANT_S && variant != SWIGLU_VARIANT_I)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown variant %d", variant);
    int st = check_gemm_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0) return ok();
    if (!A || !W_fused || !Y) return fail(SWIGLU_ERR_NULL, "A, W_fused and Y are required");
    if (!aligned16(A) || !aligned16(W_fused) || !aligned16(Y))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    const int64_t abytes = M * K * 2, ybytes = M * N * 2, wbytes = 2 * K * N * 2;
    if (overlap(Y, ybytes, A, abytes) || overlap(Y, ybytes, W_fused, wbytes))
        return fail(SWIGLU_ERR_ALIAS, "Y overlaps an input");
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const uint64_t need = swiglu::workspace_bytes_for(cus);
    if (need > kScratchBytes)
        return fail(SWIGLU_ERR_UNSUPPORTED,
                    "the device's %d compute units need %llu bytes of split-tail scratch; the "
                    "library's static scratch holds %llu", cus, (unsigned long long)need,
                    (unsigned long long)kScratchBytes);
    void *ptr = nullptr;
    st = scratch_on_device(&ptr);
    if (st != SWIGLU_OK) return st;
    const int v = variant == SWIGLU_AUTO ? swiglu_select_variant(M, N, K) : variant;
    const hipStream_t s = (hipStream_t)stream;
    if (v == SWIGLU_VARIANT_I)
        return launched(swiglu::launch_fused_interleaved(A, (int)K, W_fused, Y, (int)N, (int)M,
                                                         (int)N, (int)K,
                                                         make_ws(ptr, kScratchBytes, cus), s),
                        "fused interleaved (no-alloc)");
    return launched(swiglu::launch_fused_sequential(A, (int)K, W_fused, Y, (int)N, (int)M,
                                                    (int)N, (int)K,
                                                    make_ws(ptr, kScratchBytes, cus), s),
                    "fused sequential (no-alloc)");
}

int swiglu_unfused_ablation(const uint16_t *A, const uint16_t *W_fused, uint16_t *gate_ws,
                            uint16_t *up_ws, uint16_t *Y, int64_t M, int64_t N, int64_t K,
                            void *workspace, uint64_t workspace_bytes, void *stream) {
    int st = check_gemm_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0) return ok();
    if (!A || !W_fused || !gate_ws || !up_ws || !Y)
        return fail(SWIGLU_ERR_NULL, "A, W_fused, gate_ws, up_ws and Y are required");
    if (!aligned16(A) || !aligned16(W_fused) || !aligned16(gate_ws) || !aligned16(up_ws) ||
        !aligned16(Y))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    const int64_t abytes = M * K * 2, ybytes = M * N * 2, wbytes = 2 * K * N * 2;
    const void *outs[3] = {gate_ws, up_ws, Y};
    for (int i = 0; i < 3; ++i) {
        if (overlap(outs[i], ybytes, A, abytes) || overlap(outs[i], ybytes, W_fused, wbytes))
            return fail(SWIGLU_ERR_ALIAS, "an output overlaps an input");
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], ybytes, outs[j], ybytes))
                return fail(SWIGLU_ERR_ALIAS, "outputs overlap each other");
        if (workspace && workspace_bytes > 0 &&
            overlap(workspace, (int64_t)workspace_bytes, outs[i], ybytes))
            return fail(SWIGLU_ERR_ALIAS, "workspace overlaps an operand");
    }
    st = check_workspace(workspace, workspace_bytes);
    if (st != SWIGLU_OK) return st;
    if (workspace && workspace_bytes > 0 &&
        (overlap(workspace, (int64_t)workspace_bytes, A, abytes) ||
         overlap(workspace, (int64_t)workspace_bytes, W_fused, wbytes)))
        return fail(SWIGLU_ERR_ALIAS, "workspace overlaps an operand");
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    // the two GEMMs run in stream order, so they may share the workspace
    hipError_t e = swiglu::launch_gemm_store(A, W_fused, 0, gate_ws, (int)M, (int)N, (int)K,
                                             make_ws(workspace, workspace_bytes, cus), s);
    if (e != hipSuccess) return launched(e, "ablation gate GEMM");
    e = swiglu::launch_gemm_store(A, W_fused, 1, up_ws, (int)M, (int)N, (int)K,
                                  make_ws(workspace, workspace_bytes, cus), s);
    if (e != hipSuccess) return launched(e, "ablation up GEMM");
    return launched(swiglu::launch_silu_mul(gate_ws, up_ws, Y, M * N, s), "ablation silu_mul");
}

int swiglu_silu_mul(const uint16_t *gate, const uint16_t *up, uint16_t *Y, int64_t count,
                    void *stream) {
    if (count < 0 || count % 8 != 0)
        return fail(SWIGLU_ERR_SHAPE, "count=%lld must be a non-negative multiple of 8", (long long)count);
    if (count == 0) return ok();
    if (!gate || !up || !Y) return fail(SWIGLU_ERR_NULL, "gate, up and Y are required");
    if (!aligned16(gate) || !aligned16(up) || !aligned16(Y))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    if (overlap(Y, 2 * count, gate, 2 * count) || overlap(Y, 2 * count, up, 2 * count))
        return fail(SWIGLU_ERR_ALIAS, "Y overlaps an input");
    int st = check_device();
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_silu_mul(gate, up, Y, count, (hipStream_t)stream), "silu_mul");
}

int swiglu_pack_weights_nk(const uint16_t *W1t, const uint16_t *W2t, uint16_t *W_fused,
                           int64_t K, int64_t N, void *stream) {
    if (K < 0 || N < 0) return fail(SWIGLU_ERR_SHAPE, "negative size");
    // K is the row length of all three arrays
    if (K % 8 != 0) return fail(SWIGLU_ERR_SHAPE, "K=%lld must be a multiple of 8", (long long)K);
    if (K > kMaxK || N > kMaxN) return fail(SWIGLU_ERR_SHAPE, "size beyond limits");
    if (K == 0 || N == 0) return ok();
    if (!W1t || !W2t || !W_fused) return fail(SWIGLU_ERR_NULL, "W1t, W2t and W_fused are required");
    if (!aligned16(W1t) || !aligned16(W2t) || !aligned16(W_fused))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    const int64_t wbytes = K * N * 2;
    if (overlap(W_fused, 2 * wbytes, W1t, wbytes) || overlap(W_fused, 2 * wbytes, W2t, wbytes))
        return fail(SWIGLU_ERR_ALIAS, "W_fused overlaps W1t or W2t");
    int st = check_device();
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_pack_nk(W1t, W2t, W_fused, K, N, (hipStream_t)stream),
                    "pack_nk");
}

int swiglu_down_proj(const uint16_t *H, const uint16_t *W3t, uint16_t *Out, int64_t M, int64_t N,
                     int64_t D, void *workspace, uint64_t workspace_bytes, void *stream) {
    int st = check_down_shape(M, N, D);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || D == 0) return ok();
    if (!H || !W3t || !Out) return fail(SWIGLU_ERR_NULL, "H, W3t and Out are required");
    if (!aligned16(H) || !aligned16(W3t) || !aligned16(Out))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    const int64_t hbytes = M * N * 2, wbytes = D * N * 2, obytes = M * D * 2;
    if (overlap(Out, obytes, H, hbytes) || overlap(Out, obytes, W3t, wbytes))
        return fail(SWIGLU_ERR_ALIAS, "Out overlaps an input");
    st = check_workspace(workspace, workspace_bytes);
    if (st != SWIGLU_OK) return st;
    if (workspace && workspace_bytes > 0 &&
        (overlap(workspace, (int64_t)workspace_bytes, H, hbytes) ||
         overlap(workspace, (int64_t)workspace_bytes, W3t, wbytes) ||
         overlap(workspace, (int64_t)workspace_bytes, Out, obytes)))
        return fail(SWIGLU_ERR_ALIAS, "workspace overlaps an operand");
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_down_proj(H, W3t, Out, (int)M, (int)N, (int)D,
                                             make_ws(workspace, workspace_bytes, cus),
                                             (hipStream_t)stream),
                    "down projection");
}

int swiglu_gated_mlp(const uint16_t *A, const uint16_t *W_fused, const uint16_t *W3t,
                     uint16_t *H, uint16_t *Out, int64_t M, int64_t N, int64_t K, int variant,
                     void *workspace, uint64_t workspace_bytes, void *stream) {
    if (variant != SWIGLU_AUTO && variant != SWIGLU_VARIANT_S && variant != SWIGLU_VARIANT_I)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown variant %d", variant);
    int st = check_gemm_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    st = check_down_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return ok();   // N >= 8 and K >= 8 here (both are reduction lengths)
    const int v = variant == SWIGLU_AUTO ? swiglu_select_variant(M, N, K) : variant;
    if (!A || !W_fused || !W3t || !H || !Out)
        return fail(SWIGLU_ERR_NULL, "A, W_fused, W3t, H and Out are required");
    if (!aligned16(A) || !aligned16(W_fused) || !aligned16(W3t) || !aligned16(H) ||
        !aligned16(Out))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    const int64_t abytes = M * K * 2, wbytes = 2 * K * N * 2, w3bytes = K * N * 2;
    const int64_t hbytes = M * N * 2, obytes = M * K * 2;
    const void *ins[3] = {A, W_fused, W3t};
    const int64_t inb[3] = {abytes, wbytes, w3bytes};
    for (int i = 0; i < 3; ++i)
        if (overlap(H, hbytes, ins[i], inb[i]) || overlap(Out, obytes, ins[i], inb[i]))
            return fail(SWIGLU_ERR_ALIAS, "an output overlaps an input");
    if (overlap(H, hbytes, Out, obytes)) return fail(SWIGLU_ERR_ALIAS, "H overlaps Out");
    st = check_workspace(workspace, workspace_bytes);
    if (st != SWIGLU_OK) return st;
    if (workspace && workspace_bytes > 0) {
        for (int i = 0; i < 3; ++i)
            if (overlap(workspace, (int64_t)workspace_bytes, ins[i], inb[i]))
                return fail(SWIGLU_ERR_ALIAS, "workspace overlaps an operand");
        if (overlap(workspace, (int64_t)workspace_bytes, H, hbytes) ||
            overlap(workspace, (int64_t)workspace_bytes, Out, obytes))
            return fail(SWIGLU_ERR_ALIAS, "workspace overlaps an operand");
    }
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    const swiglu::GemmWorkspace ws = make_ws(workspace, workspace_bytes, cus);
    // the two launches run in stream order, so they may share the workspace
    hipError_t e = v == SWIGLU_VARIANT_I
                       ? swiglu::launch_fused_interleaved(A, (int)K, W_fused, H, (int)N, (int)M,
                                                          (int)N, (int)K, ws, s)
                       : swiglu::launch_fused_sequential(A, (int)K, W_fused, H, (int)N, (int)M,
                                                         (int)N, (int)K, ws, s);
    if (e != hipSuccess) return launched(e, "gated MLP: fused SwiGLU");
    return launched(swiglu::launch_down_proj(H, W3t, Out, (int)M, (int)N, (int)K, ws, s),
                    "gated MLP: down projection");
}

int swiglu_fp8_scale_exp(double amax) {
    if (!(amax > 0.0) || amax > 3.5e38) return 0;   // zero, negative, NaN or beyond float
    int e = -126;
    while (e < 126 && std::ldexp(amax, -e) > 448.0) ++e;   // smallest e: amax 2^-e <= 448
    return e;
}

int swiglu_quantize_fp8(const uint16_t *X, uint8_t *Q, int64_t count, int scale_exp,
                        void *stream) {
    if (count < 0 || count % 16 != 0)
        return fail(SWIGLU_ERR_SHAPE, "count=%lld must be a non-negative multiple of 16",
                    (long long)count);
    if (scale_exp < -126 || scale_exp > 126)
        return fail(SWIGLU_ERR_SHAPE, "scale_exp=%d outside [-126, 126]", scale_exp);
    if (count == 0) return ok();
    if (!X || !Q) return fail(SWIGLU_ERR_NULL, "X and Q are required");
    if (!aligned16(X) || !aligned16(Q))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    if (overlap(Q, count, X, 2 * count)) return fail(SWIGLU_ERR_ALIAS, "Q overlaps X");
    int st = check_device();
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_quantize_fp8(X, Q, count, scale_exp, (hipStream_t)stream),
                    "quantize_fp8");
}

int swiglu_fused_gemm_fp8(const uint8_t *A8, const uint8_t *W_fused8, uint16_t *Y, int64_t M,
                          int64_t N, int64_t K, int a_exp, int w_exp, int variant,
                          void *workspace, uint64_t workspace_bytes, void *stream) {
    if (variant != SWIGLU_AUTO && variant != SWIGLU_VARIANT_S && variant != SWIGLU_VARIANT_I)
        return fail(SWIGLU_ERR_UNSUPPORTED, "unknown variant %d", variant);
    int st = check_gemm_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (K % 16 != 0) return fail(SWIGLU_ERR_SHAPE, "K=%lld must be a multiple of 16", (long long)K);
    if (a_exp < -126 || a_exp > 126 || w_exp < -126 || w_exp > 126 || a_exp + w_exp < -126 ||
        a_exp + w_exp > 126)
        return fail(SWIGLU_ERR_SHAPE, "scale exponents out of range (a_exp + w_exp in [-126, 126])");
    if (M == 0 || N == 0) return ok();
    if (!A8 || !W_fused8 || !Y) return fail(SWIGLU_ERR_NULL, "A8, W_fused8 and Y are required");
    if (!aligned16(A8) || !aligned16(W_fused8) || !aligned16(Y))
        return fail(SWIGLU_ERR_ALIGN, "pointers must be 16-byte aligned");
    const int64_t abytes = M * K, ybytes = M * N * 2, wbytes = 2 * K * N;
    if (overlap(Y, ybytes, A8, abytes) || overlap(Y, ybytes, W_fused8, wbytes))
        return fail(SWIGLU_ERR_ALIAS, "Y overlaps an input");
    st = check_workspace(workspace, workspace_bytes);
    if (st != SWIGLU_OK) return st;
    if (workspace && workspace_bytes > 0 &&
        (overlap(workspace, (int64_t)workspace_bytes, A8, abytes) ||
         overlap(workspace, (int64_t)workspace_bytes, W_fused8, wbytes) ||
         overlap(workspace, (int64_t)workspace_bytes, Y, ybytes)))
        return fail(SWIGLU_ERR_ALIAS, "workspace overlaps an operand");
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const float scale = std::ldexp(1.0f, a_exp + w_exp);
    const int v = variant == SWIGLU_AUTO ? swiglu_select_variant(M, N, K) : variant;
    if (v == SWIGLU_VARIANT_S)
        return launched(swiglu::launch_fused_sequential_fp8(A8, W_fused8, Y, (int)M, (int)N,
                                                            (int)K, scale, (hipStream_t)stream),
                        "fused sequential fp8");
    return launched(swiglu::launch_fused_interleaved_fp8(A8, W_fused8, Y, (int)M, (int)N, (int)K,
                                                         scale,
                                                         make_ws(workspace, workspace_bytes, cus),
                                                         (hipStream_t)stream),
                    "fused interleaved fp8");
}

int swiglu_route_workspace_size(int64_t M, int64_t E, uint64_t *bytes) {
    if (!bytes) return fail(SWIGLU_ERR_NULL, "bytes is required");
    *bytes = 0;
    int st = check_route(SWIGLU_F32, M, E, 1);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    *bytes = swiglu::route_workspace_bytes(M, E, cus);
    return ok();
}

int swiglu_route(const void *logits, int logits_type, const uint8_t *valid, int32_t *ids,
                 float *weights, int32_t *counts, float *loss, int64_t M, int64_t E, int64_t k,
                 int normalize, void *workspace, uint64_t workspace_bytes, void *stream) {
    int st = check_route(logits_type, M, E, k);
    if (st != SWIGLU_OK) return st;
    const bool bf16 = logits_type == SWIGLU_BF16;
    const uint32_t size = bf16 ? 2 : 4;
    const bool none = M == 0;
    const Operand ops[] = {
        {"logits", logits, M * E * size, size, false, none},
        {"valid", valid, M, 1, false, true},
        {"ids", ids, M * k * 4, 4, true, none},
        {"weights", weights, M * k * 4, 4, true, none},
        {"counts", counts, (E + 1) * 4, 4, true, false},
        {"loss", loss, 4, 4, true, false},
        {"workspace", workspace_bytes ? workspace : nullptr, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_route(logits, bf16, valid, ids, weights, counts, loss, M, (int)E,
                                         (int)k, normalize != 0, workspace, workspace_bytes,
                                         next_arrival_tag(), cus, (hipStream_t)stream),
                    "route");
}

int swiglu_route_backward(const void *logits, int logits_type, const uint8_t *valid,
                          const int32_t *ids, const float *weights, const int32_t *counts,
                          const float *d_weights, const float *d_loss, void *d_logits, int64_t M,
                          int64_t E, int64_t k, int normalize, void *stream) {
    int st = check_route(logits_type, M, E, k);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return ok();
    const bool bf16 = logits_type == SWIGLU_BF16;
    const uint32_t size = bf16 ? 2 : 4;
    const Operand ops[] = {
        {"logits", logits, M * E * size, size, false, false},
        {"valid", valid, M, 1, false, true},
        {"ids", ids, M * k * 4, 4, false, false},
        {"weights", weights, M * k * 4, 4, false, false},
        {"counts", counts, (E + 1) * 4, 4, false, false},
        {"d_weights", d_weights, M * k * 4, 4, false, true},
        {"d_loss", d_loss, 4, 4, false, true},
        {"d_logits", d_logits, M * E * size, size, true, false},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_route_backward(logits, bf16, valid, ids, weights, counts,
                                                  d_weights, d_loss, d_logits, M, (int)E, (int)k,
                                                  normalize != 0, cus, (hipStream_t)stream),
                    "route backward");
}

int swiglu_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t slots, int64_t rank,
                               uint64_t *bytes) {
    if (!bytes) return fail(SWIGLU_ERR_NULL, "bytes is required");
    *bytes = 0;
    // the sizes of either projection: Gate and Up's K is at most 2^21, the down
    // projection's N
    int st = check_down_shape(M, N, K);
    if (st != SWIGLU_OK) st = check_gemm_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_lora(slots, 1, rank);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0 || K == 0) return ok();
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    *bytes = lora_state_bytes(M, slots, 2 * rank, swiglu::kMaxLoraCount) +
             swiglu::workspace_bytes_for(cus);
    return ok();
}

int swiglu_fused_gemm_lora(const uint16_t *X, const uint16_t *W_fused, const uint16_t *lora_a,
                           const uint16_t *lora_b, const float *lora_scale, int64_t count,
                           int64_t rank, const int32_t *ids, const float *weights, uint16_t *Y,
                           int64_t M, int64_t N, int64_t K, int64_t slots, void *workspace,
                           uint64_t workspace_bytes, void *stream) {
    int st = check_gemm_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_lora(slots, count, rank);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0) return ok();
    st = check_lora_workspace(workspace, workspace_bytes,
                              lora_state_bytes(M, slots, 2 * rank, count));
    if (st != SWIGLU_OK) return st;
    const Operand ops[] = {
        {"X", X, M * K * 2, 16, false, false},
        {"W_fused", W_fused, 2 * N * K * 2, 16, false, false},
        {"lora_a", lora_a, count * 2 * rank * K * 2, 16, false, false},
        {"lora_b", lora_b, count * 2 * N * rank * 2, 16, false, false},
        {"lora_scale", lora_scale, count * 4, 4, false, false},
        {"ids", ids, M * slots * 4, 4, false, false},
        {"weights", weights, M * slots * 4, 4, false, true},
        {"Y", Y, M * N * 2, 16, true, false},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, false},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const swiglu::LoraTable t{lora_a, lora_b, lora_scale, (int)count, (int)rank};
    return launched(lora_projection(X, W_fused, Y, M, 2 * N, K, true, t, ids, weights, slots,
                                    workspace, workspace_bytes, cus, (hipStream_t)stream),
                    "fused lora");
}

int swiglu_down_proj_lora(const uint16_t *H, const uint16_t *W3t, const uint16_t *lora_a,
                          const uint16_t *lora_b, const float *lora_scale, int64_t count,
                          int64_t rank, const int32_t *ids, const float *weights, uint16_t *Out,
                          int64_t M, int64_t N, int64_t D, int64_t slots, void *workspace,
                          uint64_t workspace_bytes, void *stream) {
    int st = check_down_shape(M, N, D);
    if (st == SWIGLU_OK) st = check_lora(slots, count, rank);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || D == 0) return ok();
    st = check_lora_workspace(workspace, workspace_bytes, lora_state_bytes(M, slots, rank, count));
    if (st != SWIGLU_OK) return st;
    const Operand ops[] = {
        {"H", H, M * N * 2, 16, false, false},
        {"W3t", W3t, D * N * 2, 16, false, false},
        {"lora_a", lora_a, count * rank * N * 2, 16, false, false},
        {"lora_b", lora_b, count * D * rank * 2, 16, false, false},
        {"lora_scale", lora_scale, count * 4, 4, false, false},
        {"ids", ids, M * slots * 4, 4, false, false},
        {"weights", weights, M * slots * 4, 4, false, true},
        {"Out", Out, M * D * 2, 16, true, false},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, false},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const swiglu::LoraTable t{lora_a, lora_b, lora_scale, (int)count, (int)rank};
    return launched(lora_projection(H, W3t, Out, M, D, N, false, t, ids, weights, slots, workspace,
                                    workspace_bytes, cus, (hipStream_t)stream),
                    "down projection lora");
}

int swiglu_gated_mlp_lora(const uint16_t *X, const uint16_t *W_fused, const uint16_t *W3t,
                          const uint16_t *gate_up_a, const uint16_t *gate_up_b,
                          const float *gate_up_scale, int64_t gate_up_count, int64_t gate_up_rank,
                          const uint16_t *down_a, const uint16_t *down_b, const float *down_scale,
                          int64_t down_count, int64_t down_rank, const int32_t *ids,
                          const float *weights, uint16_t *H, uint16_t *Out, int64_t M, int64_t N,
                          int64_t K, int64_t slots, void *workspace, uint64_t workspace_bytes,
                          void *stream) {
    int st = check_gemm_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_down_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_lora(slots, gate_up_count, gate_up_rank);
    if (st == SWIGLU_OK) st = check_lora(slots, down_count, down_rank);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return ok();
    const uint64_t need_up = lora_state_bytes(M, slots, 2 * gate_up_rank, gate_up_count);
    const uint64_t need_down = lora_state_bytes(M, slots, down_rank, down_count);
    st = check_lora_workspace(workspace, workspace_bytes, need_up > need_down ? need_up : need_down);
    if (st != SWIGLU_OK) return st;
    const Operand ops[] = {
        {"X", X, M * K * 2, 16, false, false},
        {"W_fused", W_fused, 2 * N * K * 2, 16, false, false},
        {"W3t", W3t, K * N * 2, 16, false, false},
        {"gate_up_a", gate_up_a, gate_up_count * 2 * gate_up_rank * K * 2, 16, false, false},
        {"gate_up_b", gate_up_b, gate_up_count * 2 * N * gate_up_rank * 2, 16, false, false},
        {"gate_up_scale", gate_up_scale, gate_up_count * 4, 4, false, false},
        {"down_a", down_a, down_count * down_rank * N * 2, 16, false, false},
        {"down_b", down_b, down_count * K * down_rank * 2, 16, false, false},
        {"down_scale", down_scale, down_count * 4, 4, false, false},
        {"ids", ids, M * slots * 4, 4, false, false},
        {"weights", weights, M * slots * 4, 4, false, true},
        {"H", H, M * N * 2, 16, true, false},
        {"Out", Out, M * K * 2, 16, true, false},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, false},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    const swiglu::LoraTable up{gate_up_a, gate_up_b, gate_up_scale, (int)gate_up_count,
                               (int)gate_up_rank};
    const swiglu::LoraTable down{down_a, down_b, down_scale, (int)down_count, (int)down_rank};
    // the launches run in stream order, so they share the workspace
    const hipError_t e = lora_projection(X, W_fused, H, M, 2 * N, K, true, up, ids, weights, slots,
                                         workspace, workspace_bytes, cus, s);
    if (e != hipSuccess) return launched(e, "gated MLP lora: fused SwiGLU");
    return launched(lora_projection(H, W3t, Out, M, K, N, false, down, ids, weights, slots,
                                    workspace, workspace_bytes, cus, s),
                    "gated MLP lora: down projection");
}

int swiglu_fused_gemm_train(const uint16_t *A, const uint16_t *W_fused, uint16_t *H, uint16_t *GU,
                            int64_t M, int64_t N, int64_t K, void *workspace,
                            uint64_t workspace_bytes, void *stream) {
    int st = check_train_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0) return ok();
    const Operand ops[] = {
        {"A", A, M * K * 2, 16, false, false},
        {"W_fused", W_fused, 2 * N * K * 2, 16, false, false},
        {"H", H, M * N * 2, 16, true, false},
        {"GU", GU, 2 * M * N * 2, 16, true, false},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_fused_train(A, W_fused, H, GU, (int)M, (int)N, (int)K,
                                               make_ws(workspace, workspace_bytes, cus),
                                               (hipStream_t)stream),
                    "fused training forward");
}

int swiglu_gated_mlp_train(const uint16_t *A, const uint16_t *W_fused, const uint16_t *W3t,
                           uint16_t *H, uint16_t *GU, uint16_t *Out, int64_t M, int64_t N,
                           int64_t K, void *workspace, uint64_t workspace_bytes, void *stream) {
    int st = check_train_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_down_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return ok();
    const Operand ops[] = {
        {"A", A, M * K * 2, 16, false, false},
        {"W_fused", W_fused, 2 * N * K * 2, 16, false, false},
        {"W3t", W3t, K * N * 2, 16, false, false},
        {"H", H, M * N * 2, 16, true, false},
        {"GU", GU, 2 * M * N * 2, 16, true, false},
        {"Out", Out, M * K * 2, 16, true, false},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    const swiglu::GemmWorkspace ws = make_ws(workspace, workspace_bytes, cus);
    const hipError_t e =
        swiglu::launch_fused_train(A, W_fused, H, GU, (int)M, (int)N, (int)K, ws, s);
    if (e != hipSuccess) return launched(e, "gated MLP training forward: fused SwiGLU");
    return launched(swiglu::launch_down_train(H, W3t, Out, (int)M, (int)N, (int)K, ws, s),
                    "gated MLP training forward: down projection");
}

int swiglu_down_proj_backward(const uint16_t *dOut, const uint16_t *H, const uint16_t *W3t,
                              uint16_t *dH, void *dW3t, const void *dW3t_add, int grad_type,
                              int64_t M, int64_t N, int64_t D, void *workspace,
                              uint64_t workspace_bytes, void *stream) {
    int st = check_grad_type(grad_type);
    if (st == SWIGLU_OK) st = check_down_backward_shape(M, N, D);
    if (st != SWIGLU_OK) return st;
    if (!dH && !dW3t) return fail(SWIGLU_ERR_NULL, "dH or dW3t is required");
    if (dW3t_add && !dW3t) return fail(SWIGLU_ERR_NULL, "dW3t_add without dW3t");
    const bool none = M == 0;
    const Operand ops[] = {
        {"dOut", dOut, M * D * 2, 16, false, none},
        {"H", H, M * N * 2, 16, false, none || !dW3t},
        {"W3t", W3t, D * N * 2, 16, false, none || !dH},
        {"dW3t_add", add_operand(dW3t_add, dW3t), D * N * grad_size(grad_type), 16, false, true},
        {"dH", dH, M * N * 2, 16, true, true},
        {"dW3t", dW3t, D * N * grad_size(grad_type), 16, true, true},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    return launched(swiglu::launch_down_backward(dOut, H, W3t, dH, dW3t, dW3t_add,
                                                 grad_type == SWIGLU_F32, (int)M, (int)N, (int)D,
                                                 make_ws(workspace, workspace_bytes, cus), s),
                    "down projection backward");
}

int swiglu_fused_gemm_backward(const uint16_t *dH, const uint16_t *A, const uint16_t *W_fused,
                               const uint16_t *GU, uint16_t *dGU, uint16_t *dA, void *dW_fused,
                               const void *dW_fused_add, int grad_type, int64_t M, int64_t N,
                               int64_t K, void *workspace, uint64_t workspace_bytes,
                               void *stream) {
    int st = check_grad_type(grad_type);
    if (st == SWIGLU_OK) st = check_stage_backward_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (dW_fused_add && !dW_fused) return fail(SWIGLU_ERR_NULL, "dW_fused_add without dW_fused");
    const bool none = M == 0;
    const int64_t weight = 2 * N * K;
    const Operand ops[] = {
        {"dH", dH, M * N * 2, 16, false, none},
        {"A", A, M * K * 2, 16, false, none || !dW_fused},
        {"W_fused", W_fused, weight * 2, 16, false, none || !dA},
        {"GU", GU == dGU ? nullptr : GU, 2 * M * N * 2, 16, false, none || GU == dGU},
        {"dW_fused_add", add_operand(dW_fused_add, dW_fused), weight * grad_size(grad_type), 16,
         false, true},
        {"dGU", dGU, 2 * M * N * 2, 16, true, none},
        {"dA", dA, M * K * 2, 16, true, true},
        {"dW_fused", dW_fused, weight * grad_size(grad_type), 16, true, true},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    if (M > 0) e = swiglu::launch_gate_grad(dH, GU, dGU, M * N, s);
    if (e == hipSuccess)
        e = swiglu::launch_stage_backward(dGU, A, W_fused, dA, dW_fused, dW_fused_add,
                                          grad_type == SWIGLU_F32, (int)M, (int)N, (int)K,
                                          make_ws(workspace, workspace_bytes, cus), s);
    return launched(e, "fused SwiGLU backward");
}

int swiglu_gated_mlp_backward(const uint16_t *dOut, const uint16_t *A, const uint16_t *W_fused,
                              const uint16_t *W3t, const uint16_t *H, const uint16_t *GU,
                              uint16_t *dGU, uint16_t *dA, void *dW_fused,
                              const void *dW_fused_add, void *dW3t, const void *dW3t_add,
                              int grad_type, int64_t M, int64_t N, int64_t K, void *workspace,
                              uint64_t workspace_bytes, void *stream) {
    int st = check_grad_type(grad_type);
    if (st == SWIGLU_OK) st = check_block_backward_shape(M, N, K);
    if (st != SWIGLU_OK) return st;
    if (dW_fused_add && !dW_fused) return fail(SWIGLU_ERR_NULL, "dW_fused_add without dW_fused");
    if (dW3t_add && !dW3t) return fail(SWIGLU_ERR_NULL, "dW3t_add without dW3t");
    const bool none = M == 0;
    const int64_t weight = 2 * N * K, size = grad_size(grad_type);
    const Operand ops[] = {
        {"dOut", dOut, M * K * 2, 16, false, none},
        {"A", A, M * K * 2, 16, false, none || !dW_fused},
        {"W_fused", W_fused, weight * 2, 16, false, none || !dA},
        {"W3t", W3t, weight, 16, false, none},
        {"H", H, M * N * 2, 16, false, none || !dW3t},
        {"GU", GU == dGU ? nullptr : GU, 2 * M * N * 2, 16, false, none || GU == dGU},
        {"dW_fused_add", add_operand(dW_fused_add, dW_fused), weight * size, 16, false, true},
        {"dW3t_add", add_operand(dW3t_add, dW3t), N * K * size, 16, false, true},
        {"dGU", dGU, 2 * M * N * 2, 16, true, none},
        {"dA", dA, M * K * 2, 16, true, true},
        {"dW_fused", dW_fused, weight * size, 16, true, true},
        {"dW3t", dW3t, N * K * size, 16, true, true},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    swiglu::GemmWorkspace ws = make_ws(workspace, workspace_bytes, cus);
    const bool f32 = grad_type == SWIGLU_F32;
    hipError_t e = swiglu::launch_gate_backward(dOut, H, W3t, GU, dGU, dW3t, dW3t_add, f32, (int)M,
                                                (int)N, (int)K, ws, s);
    ws.tag = next_arrival_tag();
    if (e == hipSuccess)
        e = swiglu::launch_stage_backward(dGU, A, W_fused, dA, dW_fused, dW_fused_add, f32, (int)M,
                                          (int)N, (int)K, ws, s);
    return launched(e, "gated MLP backward");
}

int swiglu_quantize_mx4(const uint16_t *X, uint8_t *Q, uint8_t *S, int64_t rows, int64_t K,
                        void *stream) {
    int st = check_mx4_matrix(rows, K);
    if (st != SWIGLU_OK) return st;
    if (rows == 0) return ok();
    const Operand ops[] = {
        {"X", X, rows * K * 2, 16, false, false},
        {"Q", Q, rows * K / 2, 16, true, false},
        {"S", S, rows * K / 32, 1, true, false},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st == SWIGLU_OK) st = check_device();
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_quantize_mx4(X, Q, S, rows * K, (hipStream_t)stream),
                    "4-bit quantizer");
}

int swiglu_dequantize_mx4(const uint8_t *Q, const uint8_t *S, uint16_t *X, int64_t rows, int64_t K,
                          void *stream) {
    int st = check_mx4_matrix(rows, K);
    if (st != SWIGLU_OK) return st;
    if (rows == 0) return ok();
    const Operand ops[] = {
        {"Q", Q, rows * K / 2, 16, false, false},
        {"S", S, rows * K / 32, 1, false, false},
        {"X", X, rows * K * 2, 16, true, false},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st == SWIGLU_OK) st = check_device();
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_dequantize_mx4(Q, S, X, rows * K, (hipStream_t)stream),
                    "4-bit dequantizer");
}

int swiglu_fused_gemm_mx4(const uint16_t *A, const uint8_t *Wq, const uint8_t *Ws, uint16_t *Y,
                          int64_t M, int64_t N, int64_t K, void *workspace,
                          uint64_t workspace_bytes, void *stream) {
    int st = check_gemm_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_mx4_groups("K", K);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || N == 0) return ok();
    const Operand ops[] = {
        {"A", A, M * K * 2, 16, false, false},
        {"Wq", Wq, N * K, 16, false, false},
        {"Ws", Ws, N * K / 16, 4, false, false},
        {"Y", Y, M * N * 2, 16, true, false},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_fused_mx4(A, Wq, Ws, Y, (int)M, (int)N, (int)K,
                                             make_ws(workspace, workspace_bytes, cus),
                                             (hipStream_t)stream),
                    "fused 4-bit");
}

int swiglu_down_proj_mx4(const uint16_t *H, const uint8_t *W3q, const uint8_t *W3s, uint16_t *Out,
                         int64_t M, int64_t N, int64_t D, void *workspace,
                         uint64_t workspace_bytes, void *stream) {
    int st = check_down_shape(M, N, D);
    if (st == SWIGLU_OK) st = check_mx4_groups("N", N);
    if (st != SWIGLU_OK) return st;
    if (M == 0 || D == 0) return ok();
    const Operand ops[] = {
        {"H", H, M * N * 2, 16, false, false},
        {"W3q", W3q, D * N / 2, 16, false, false},
        {"W3s", W3s, D * N / 32, 4, false, false},
        {"Out", Out, M * D * 2, 16, true, false},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    return launched(swiglu::launch_down_proj_mx4(H, W3q, W3s, Out, (int)M, (int)N, (int)D,
                                                 make_ws(workspace, workspace_bytes, cus),
                                                 (hipStream_t)stream),
                    "down projection 4-bit");
}

int swiglu_gated_mlp_mx4(const uint16_t *A, const uint8_t *Wq, const uint8_t *Ws,
                         const uint8_t *W3q, const uint8_t *W3s, uint16_t *H, uint16_t *Out,
                         int64_t M, int64_t N, int64_t K, void *workspace,
                         uint64_t workspace_bytes, void *stream) {
    int st = check_gemm_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_down_shape(M, N, K);
    if (st == SWIGLU_OK) st = check_mx4_groups("K", K);
    if (st == SWIGLU_OK) st = check_mx4_groups("N", N);
    if (st != SWIGLU_OK) return st;
    if (M == 0) return ok();
    const Operand ops[] = {
        {"A", A, M * K * 2, 16, false, false},
        {"Wq", Wq, N * K, 16, false, false},
        {"Ws", Ws, N * K / 16, 4, false, false},
        {"W3q", W3q, K * N / 2, 16, false, false},
        {"W3s", W3s, K * N / 32, 4, false, false},
        {"H", H, M * N * 2, 16, true, false},
        {"Out", Out, M * K * 2, 16, true, false},
        {"workspace", workspace, (int64_t)workspace_bytes, 256, true, true},
    };
    st = check_operands(ops, sizeof ops / sizeof ops[0]);
    if (st != SWIGLU_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != SWIGLU_OK) return st;
    const hipStream_t s = (hipStream_t)stream;
    const swiglu::GemmWorkspace ws = make_ws(workspace, workspace_bytes, cus);
    const hipError_t e = swiglu::launch_fused_mx4(A, Wq, Ws, H, (int)M, (int)N, (int)K, ws, s);
    if (e != hipSuccess) return launched(e, "gated MLP 4-bit: fused SwiGLU");
    return launched(swiglu::launch_down_proj_mx4(H, W3q, W3s, Out, (int)M, (int)N, (int)K, ws, s),
                    "gated MLP 4-bit: down projection");
}

}  // extern "C"
