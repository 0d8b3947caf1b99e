// Launchers of the drafted-tree operators (rotary positions, cache write and read, tree attention).
#pragma once
#include <mutex>
#include <utility>

#include "common.cuh"

namespace af {

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Launch with programmatic stream serialization: the kernel may start before its predecessor in the stream is done and
// waits for it (griddepcontrol.wait) before it touches memory.  A kernel that may write a cache (rows, keys that move, slots
// read back as the fp32 cache of a kv head) does not launch its dependents early, and its stores are visible before it ends:
// the decode attention reads all but the last slot before its own wait, so it would see the cache as it was.
template <typename K, typename... A>
cudaError_t launch_chained(K kernel, dim3 grid, int threads, int smem, cudaStream_t s, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// A kernel's opt-in to more than 48 KB of dynamic shared memory, once per device.
struct SmemOptIn {
    std::mutex mu;
    bool done[kMaxDevices] = {};
    cudaError_t operator()(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e) return e;
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        std::lock_guard<std::mutex> lk(mu);
        if (done[dev]) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (!e) done[dev] = true;
        return e;
    }
};

// ---- rotary positions (rope.cu)
constexpr int kRopeMaxPairs = 128;  // head_dim <= 256

// Angle per position of each pair as a fraction of a turn in 64-bit fixed point: position times turn, wrapped
// to 64 bits, is the angle modulo one turn, for any int32 position and without fp64 on the device.
struct RopeTurns {
    uint64_t turn[kRopeMaxPairs];
};
struct RopeArgs {
    const void* x = nullptr;
    void* y = nullptr;
    int64_t ldx = 0, ldy = 0;
    int f16 = 0, n = 0, heads = 0, D = 0, R = 0, half = 0;
    const int* pos = nullptr;  // nullable: position of row r is pos0 + r
    int pos0 = 0;
    float mag = 1.f;
};
cudaError_t launch_rope(const RopeArgs& a, const RopeTurns& t, cudaStream_t s);

// ---- cache rows (kv_rows.cu)
struct KvRows {
    void* k = nullptr;  // [KVH][ctx][D] values, or codes (kv_code_bytes per slot)
    void* v = nullptr;
    __half* ks = nullptr;  // [KVH][ctx][D / 32] scales of a quantized cache
    __half* vs = nullptr;
    int type = 0;  // af_dtype
    int KVH = 0, D = 0, ctx = 0;
};
cudaError_t launch_kv_write(const KvRows& c, const float* k, const float* v, int64_t ld, int n, const int* slots,
                            int slot0, cudaStream_t s);
cudaError_t launch_kv_read(const KvRows& c, int n, const int* slots, int slot0, float* k, float* v, int64_t ld,
                           cudaStream_t s);

// ---- tree attention (attn_tree.cu)
constexpr int kTreeMax = 1024;  // nodes
cudaError_t launch_tree_mask(const int* parent, int n, int pos0, unsigned* mask, int* pos, cudaStream_t s);

struct TreeArgs {
    const float* q = nullptr;
    int64_t ldq = 0;
    KvRows c;
    int H = 0, past = 0, n = 0;
    const unsigned* mask = nullptr;
    float* out = nullptr;
    int64_t ldo = 0;
    float* ws = nullptr;
};
// What a row's sums are multiplied with: one over the sum of its weights; where that is 0, 0 for a row that sees no slot, and
// NaN for one that sees some, whose scores are all -infinity.
__device__ __forceinline__ float row_inverse(const TreeArgs& a, int node, float sum) {
    if (sum != 0.f) return 1.f / sum;
    bool sees = a.past > 0;
    const int words = (a.n + 31) / 32;
    for (int w = 0; w < words && !sees; w++)
        sees = (__ldcg(a.mask + (int64_t)node * words + w) & (w == words - 1 && a.n % 32 ? (1u << (a.n % 32)) - 1u : ~0u)) != 0;
    return sees ? __uint_as_float(0x7FC00000u) : 0.f;
}
// A call with many rows goes to the tcgen05 kernel (attn_tree_tc.cu): its 64-slot tiles and splits; splits = 0: not.
struct TreeTcPlan {
    int tiles = 0, splits = 0;
};
TreeTcPlan tree_tc_plan(int H, int KVH, int D, int type, int past, int n);
// Writes the workspace's parts [0, splits), or the output where there is one.
cudaError_t launch_attn_tree_tc(const TreeArgs& a, const TreeTcPlan& p, cudaStream_t s);

size_t attn_tree_ws_bytes(int H, int KVH, int D, int type, int past, int n);
cudaError_t launch_attn_tree(const TreeArgs& a, cudaStream_t s);

}  // namespace af
