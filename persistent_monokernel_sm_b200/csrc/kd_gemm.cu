// kd_gemm.cu -- the batched products of a layer on the 5th-generation tensor cores: linear
// (bias, activation, residual in the epilogue), the gated feed-forward block and its gradients.
//
// One kernel computes D[n][t] = sum_k A[n][k] B[t][k]: A is the weight side, whose index n is
// the contiguous one of the output, B the token side. Tensor memory then holds an output
// feature per lane and a token per column, so that
//  * a bias is one register per thread, and 32 lanes write 32 neighbouring outputs of a token;
//  * few tokens (one, at serving) cost few columns: the tile is 128 features x 16 tokens there,
//    and the tensor core streams weights at the rate of HBM;
//  * the gated block's gate and up rows of one feature lie 16 lanes apart (its A tile takes 16
//    gate rows, 16 up rows, 16 gate rows ...), so act(g) * u is one shuffle per column pair.
//
// Structure: one CTA per SM loops over output tiles. A producer thread fills a ring of 64-deep
// k-blocks by TMA (128-byte swizzle), one thread issues tcgen05.mma, eight warps read the
// accumulators out of tensor memory, which holds two tiles so that the products of the next one
// run meanwhile, and write the output through shared memory by TMA. Wide tiles are done by two
// CTAs at once (cta_group::2: 256 features, each CTA loads half of the tokens' operand). With few tiles the reduction
// is split over the CTAs of a cluster, whose partial tiles are summed in rank order through
// distributed shared memory: no workspace, one launch, the same result every time. One to four
// tokens against a weight with rows over k go to row_kernel, without the tensor cores.
//
// What bounds it: with many tokens the tensor cores (4,096 x 14,336 x 4,096 with both gated
// projections: 596 us alone, 1.61 of the measured 1.63 PFLOP/s; in a loop of seconds the power cap,
// 714 us, 1.35 of 1.38); with one token HBM (128,256 x 4,096: 151 us in a graph over two weights in turn,
// 7.0 TB/s of reads alone, where the measured 6.5 is a copy's; 158 to 177 called one by one, by the box);
// between them what a tile costs besides its products: start, ring fill, epilogue, exchange, 3.7 us for the
// smallest call.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <type_traits>

#include "kd.h"
#include "kd_layout.h"
#include "kd_ops.h"
#include "kd_sm100.h"

namespace kd {

// ------------------------------------------------------------------ host helpers
static thread_local char t_err[512];

int op_fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_err, sizeof t_err, fmt, ap);
    va_end(ap);
    return code;
}

int op_sm_count(int* sms) {
    static std::atomic<int> cached[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return op_fail(KD_ECUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    int n = dev < 64 ? cached[dev].load() : 0;
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return op_fail(KD_ECUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
        if (dev < 64) cached[dev].store(n);
    }
    *sms = n;
    return KD_OK;
}

static thread_local long long t_limit_ns = 2000000000ll;
OpWaits own_waits() { return {op_clocks(t_limit_ns), nullptr}; }

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load();
    if (!f) {
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &st) != cudaSuccess ||
            st != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f);
    }
    return (EncodeFn)f;
}

static int encode(CUtensorMap* m, int dtype, const void* base, int rank, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, bool swizzle = true) {
    EncodeFn f = encode_fn();
    if (!f) return op_fail(KD_ECUDA, "the driver has no cuTensorMapEncodeTiled");
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUtensorMapDataType type = dtype == KD_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == KD_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    auto fill = [&]() {
        return f(m, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = fill();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // The driver's function needs a current context, which a host thread gets with its first runtime
        // call of some kinds; this may be the thread's first.
        int dev = 0;
        if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = fill();
    }
    if (r != CUDA_SUCCESS) return op_fail(KD_ECUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return KD_OK;
}

int make_map_2d(CUtensorMap* m, int dtype, const void* base, int64_t cols, int64_t rows, int64_t ld, int box_cols,
                int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    return encode(m, dtype, base, 2, dims, strides, box);
}

// Of an output: boxes as they lie in shared memory, without a swizzle.
static int make_map_out(CUtensorMap* m, int dtype, const void* base, int64_t cols, int64_t rows, int64_t ld,
                        int box_cols, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * (dtype == KD_F32 ? 4 : 2)};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    return encode(m, dtype, base, 2, dims, strides, box, false);
}

int make_map_3d(CUtensorMap* m, int dtype, const void* base, int64_t c0, int64_t c1, int64_t c2, int64_t ld1,
                int64_t ld2, int box0, int box1, int box2) {
    const cuuint64_t dims[3] = {(cuuint64_t)c0, (cuuint64_t)c1, (cuuint64_t)c2};
    const cuuint64_t strides[2] = {(cuuint64_t)ld1 * 2, (cuuint64_t)ld2 * 2};
    const cuuint32_t box[3] = {(cuuint32_t)box0, (cuuint32_t)box1, (cuuint32_t)box2};
    return encode(m, dtype, base, 3, dims, strides, box);
}

namespace {

// Three warpgroups: two of epilogue warps, one with the producer's and the issuer's warp. The
// epilogue takes registers from the third: 256 x 216 + 128 x 72 = 384 x 168, the launch's total.
constexpr int kGemmThreads = 384;
constexpr int kEpiRegs = 216, kAuxRegs = 72;
// An accumulator of the tensor cores is truncated towards zero at every step of 16 products. Measured,
// relative: 9.8e-8 a step where all terms have one sign (1e-3 over 2^17 products), 1.7e-8 where signs are
// mixed (4.3e-6 at k = 4,096). Where the result is kept in fp32, sums of more than 512 products are
// therefore taken as several, added in registers with rounding to nearest. A result of 16 bits does not
// show it until its sum is long: the same is done for it from 2^15 products of a CTA in fp16 and 2^18 in
// bf16 on, where the truncation could reach 0.41 of the type's half step (2^-11, 2^-8).
constexpr int kChunk = 8;                        // 64-deep k-blocks
constexpr int kLongF16 = 512, kLongBF16 = 4096;  // k-blocks
constexpr int kBK = 64;            // k-block: 128 bytes of a row
constexpr int kABytes = 128 * kBK * 2;
constexpr int kMaxRing = 12;
// Columns of a tile from which CTAs work in pairs (us, single CTAs and pairs, in a loop of seconds): 256
// columns, the gated block of 4,096 x 4,096 x 14,336 758 / 714, 500 x 2,048 x 8,192 40.1 / 37.9; 128 columns,
// 1,024 x 2,048 x 2,048 13.2 / 13.8.
constexpr int kPairMin = 192;
constexpr int kRingBytes = 192 * 1024;
// Behind the ring: 4 KB for each epilogue warp, two halves in turn, from which TMA writes the
// output. A column of the accumulator is then one store to shared memory, with no address to
// compute; stored to global memory from the lanes it took 28 instructions, and a 128 x 256 tile
// 9 us where its products take 13 (at k = 2,048).
constexpr int kStageBytes = 4096;
constexpr int kSmemBytes = 1024 + kRingBytes + 8 * kStageBytes;
constexpr int kGroup = 8;  // token tiles that are taken together while the weight tiles advance

// Which index of the two operands is the contiguous one in memory: k of both; the feature of A
// and k of B (a transposed weight); the feature and the token (a sum over rows).
enum { LAY_KK = 0, LAY_MK = 1, LAY_MM = 2 };
enum { EPI_LINEAR = 0, EPI_GATED = 1, EPI_GATED_BWD = 2 };

struct GemmArgs {
    int n_tiles, t_tiles;  // tiles over features and tokens
    int kb0, kb;           // k-blocks of the first operand pair, of both
    int bn, stages, splits;
    uint32_t idesc;
    int act;
    int64_t N, M;  // features (of the output), tokens
    const void* bias;
    const void* res;  // residual; the backward pass's dh
    int64_t ld_res;
    void* out;
    void* out2;  // the backward pass's du; the second of two products of one A (t_half > 0)
    int64_t ld_out, ld_out2;
    int tma_out;  // outputs by TMA (aligned rows), else from the lanes
    // This launch needs nothing of the one before it, only of those before that, which that one has
    // waited for: it starts beside it, and waits for its end before its own.
    int beside;
    int t_half;  // token tiles of the first of two products with the same A; 0: one product
    OpWaits waits;
};

// ------------------------------------------------------------------ activations
// fp32 throughout. silu and its slope take the fast exponential, which is off by 2 + 1.2 |z| units in the
// last place: 26 at z = -20, 1.5e-6 of a silu of -4e-8; towards z > 0 it fades, e^-z being small beside 1.
// gelu's 1 + erf loses its leading digits for z << 0: it is good to 2^-23 |z|, not to digits of a value that
// is smaller than that.
template <int ACT>
__device__ __forceinline__ float act_fn(float z) {
    if constexpr (ACT == KD_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
    if constexpr (ACT == KD_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
    if constexpr (ACT == KD_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    return z;
}
template <int ACT>
__device__ __forceinline__ void act_slope(float z, float* a, float* s) {
    if constexpr (ACT == KD_ACT_RELU) {
        *a = z > 0.f ? z : (z != z ? z : 0.f);
        *s = z > 0.f ? 1.f : 0.f;
    } else if constexpr (ACT == KD_ACT_SILU) {
        const float p = __fdividef(1.f, 1.f + __expf(-z));
        *a = z * p;
        *s = p * (1.f + z * (1.f - p));
    } else if constexpr (ACT == KD_ACT_GELU) {
        const float c = 0.5f * (1.f + erff(z * 0.70710678118654752f));
        *a = z * c;
        *s = c + z * 0.39894228040143268f * __expf(-0.5f * z * z);
    } else {
        *a = z;
        *s = 1.f;
    }
}

// ------------------------------------------------------------------ epilogue
template <typename T> __device__ __forceinline__ float to_f(T v) { return Half2<T>::up(v); }
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f(float v) { return Half2<T>::down(v); }
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }

// A warp's way out of the accumulators.
struct Out {
    const CUtensorMap *o0, *o1;
    uint8_t* stage;  // this warp's 4 KB of shared memory
    int flip;        // the half that is used next
    int quad, lane;
};

// Rows (tokens) of a box: two boxes of 16 fp32 columns, one of 32 of 16 bits.
template <int COLS, typename O> struct Box { static constexpr int rows = sizeof(O) == 4 || COLS < 32 ? 16 : 32; };

// Only boxes whose columns all exist go this way: TMA writes whole 16 bytes, also past the end of
// a row that is no multiple of them (rows of a box past the last token are left out exactly).

// The half of the stage that the store before the last has left; then, once the warp has filled
// it, its way to global memory.
__device__ __forceinline__ uint8_t* stage_open(Out& w) {
    if (w.lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    uint8_t* p = w.stage + w.flip * (kStageBytes / 2);
    w.flip ^= 1;
    return p;
}
__device__ __forceinline__ void stage_store(const Out& w, const CUtensorMap* m, const uint8_t* from, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m), "r"(x), "r"(y),
                 "r"(smem_u32(from))
                 : "memory");
}
__device__ __forceinline__ void stage_fence() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// COLS columns (tokens t0 ...) of this warp's 32 lanes; w.quad: which 32 rows of the tile.
template <int EPI, int ACT, int COLS, typename T, typename O>
__device__ __forceinline__ void emit(const GemmArgs& g, Out& w, const float* v, int tile_n, int64_t t0, float bias,
                                     bool second, const float* given) {
    const int lane = w.lane;
    if constexpr (EPI == EPI_LINEAR) {
        const int n0 = tile_n * 128 + w.quad * 32, n = n0 + lane;
        if (n0 >= g.N) return;
        const int left = n < g.N ? (int)min((int64_t)COLS, g.M - t0) : 0;  // columns that exist
        float r[COLS];
        if (COLS == 2) {
#pragma unroll
            for (int j = 0; j < COLS; ++j) r[j] = act_fn<ACT>(v[j] + bias) + given[j];
        } else if (g.res) {
            const O* res = (const O*)g.res + t0 * g.ld_res + n;
#pragma unroll
            for (int j = 0; j < COLS; ++j, res += g.ld_res) r[j] = j < left ? to_f<O>(*res) : 0.f;
#pragma unroll
            for (int j = 0; j < COLS; ++j) r[j] = act_fn<ACT>(v[j] + bias) + r[j];
        } else {
#pragma unroll
            for (int j = 0; j < COLS; ++j) r[j] = act_fn<ACT>(v[j] + bias);
        }
        if (COLS >= 16 && g.tma_out && n0 + 32 <= g.N) {
            constexpr int R = Box<COLS, O>::rows;
#pragma unroll
            for (int c = 0; c < COLS; c += R) {
                uint8_t* p = stage_open(w);
                O* q = reinterpret_cast<O*>(p) + lane;
#pragma unroll
                for (int j = 0; j < R; ++j) q[j * 32] = from_f<O>(r[c + j]);
                stage_fence();
                if (lane == 0 && t0 + c < g.M) stage_store(w, second ? w.o1 : w.o0, p, n0, (int)t0 + c);
                if (lane == 0) stage_commit();
            }
        } else {
            const int64_t ld = second ? g.ld_out2 : g.ld_out;
            O* out = (O*)(second ? g.out2 : g.out) + t0 * ld + n;
#pragma unroll
            for (int j = 0; j < COLS; ++j, out += ld)
                if (j < left) *out = from_f<O>(r[j]);
        }
    } else {
        // Lanes 0-15 hold gate rows, 16-31 the up rows of the same features: of columns 2j and
        // 2j + 1 the lower lanes finish the first, the upper ones the second.
        const bool low = lane < 16;
        const int n0 = tile_n * 64 + w.quad * 16, n = n0 + (lane & 15);
        if (n0 >= g.N) return;
        const int64_t at = t0 + (low ? 0 : 1);
        const int left = n < g.N ? (int)min((int64_t)COLS, g.M - at) : 0;
        T dh[COLS / 2];
        if constexpr (EPI == EPI_GATED_BWD) {
            const T* p = (const T*)g.res + at * g.ld_res + n;
#pragma unroll
            for (int j = 0; j < COLS; j += 2, p += 2 * g.ld_res) dh[j / 2] = j < left ? *p : from_f<T>(0.f);
        }
        const bool staged = COLS >= 16 && g.tma_out && n0 + 16 <= g.N;
        uint8_t* p = staged ? stage_open(w) : nullptr;
        T *q0 = reinterpret_cast<T*>(p) + lane, *q1 = q0 + 512;  // [token][16 features]: 32 lanes, two rows
        const int64_t ld = g.ld_out;
        T *out = (T*)g.out + at * ld + n, *out2 = (T*)g.out2 + at * ld + n;
#pragma unroll
        for (int j = 0; j < COLS; j += 2) {
            const float got = __shfl_xor_sync(0xffffffffu, low ? v[j + 1] : v[j], 16);
            const float gate = low ? v[j] : got, up = low ? got : v[j + 1];
            float a, b = 0.f;
            if constexpr (EPI == EPI_GATED) {
                a = act_fn<ACT>(gate) * up;
            } else {
                float f, s;
                act_slope<ACT>(gate, &f, &s);
                const float d = to_f<T>(dh[j / 2]);
                a = d * up * s, b = d * f;
            }
            if (staged) {
                q0[j * 16] = from_f<T>(a);
                if constexpr (EPI == EPI_GATED_BWD) q1[j * 16] = from_f<T>(b);
            } else {
                if (j < left) {
                    *out = from_f<T>(a);
                    if constexpr (EPI == EPI_GATED_BWD) *out2 = from_f<T>(b);
                }
                out += 2 * ld;
                if constexpr (EPI == EPI_GATED_BWD) out2 += 2 * ld;
            }
        }
        if (staged) {
            stage_fence();
            if (lane == 0 && t0 < g.M) {
                stage_store(w, w.o0, p, n0, (int)t0);
                if constexpr (EPI == EPI_GATED_BWD) stage_store(w, w.o1, p + 1024, n0, (int)t0);
            }
            if (lane == 0) stage_commit();
        }
    }
}

template <int EPI, int LAY, int COLS, typename T, typename O>
__device__ __forceinline__ void emit_act(const GemmArgs& g, Out& w, const float* v, int tile_n, int64_t t0, float bias,
                                         bool second, const float* given = nullptr) {
    switch (LAY == LAY_MM ? KD_ACT_NONE : g.act) {
        case KD_ACT_RELU: emit<EPI, KD_ACT_RELU, COLS, T, O>(g, w, v, tile_n, t0, bias, second, given); break;
        case KD_ACT_SILU: emit<EPI, KD_ACT_SILU, COLS, T, O>(g, w, v, tile_n, t0, bias, second, given); break;
        case KD_ACT_GELU: emit<EPI, KD_ACT_GELU, COLS, T, O>(g, w, v, tile_n, t0, bias, second, given); break;
        default: emit<EPI, KD_ACT_NONE, COLS, T, O>(g, w, v, tile_n, t0, bias, second, given); break;
    }
}

// ------------------------------------------------------------------ the kernel
// Where a wait of a CTA or of its pair has given up and no thread starts anything any more, products and
// copies may still be under way, whichever role gave up. They end before the shared and the tensor memory
// goes: the products by a commit (on both CTAs of a pair), the copies on their barriers; of a pair, where
// one CTA may have loaded what the other has not, by a pause. Not inlined, which
// leaves the code out of the way: 0.1 us a launch less.
template <int CG>
__device__ __noinline__ void unwind_products(bool first, uint32_t drain) {
    if (first) {
        if constexpr (CG == 2) tc_commit_pair(drain);
        else tc_commit(drain);
    }
    mbar_drain(drain, 0);
}
template <int CG>
__device__ __noinline__ void unwind_loads(uint32_t full, int stages, int loads) {
    if constexpr (CG == 2) {
        drain_pause();
    } else {
        for (int i = loads > stages ? loads - stages : 0; i < loads; ++i) mbar_drain(full + 8 * (i % stages), (i / stages) & 1);
    }
}

// LONG: a 16-bit result of a sum that is taken as several.
template <int CG, int EPI, int LAY, typename T, typename O, bool LONG>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap a1,
                const __grid_constant__ CUtensorMap b0, const __grid_constant__ CUtensorMap b1,
                const __grid_constant__ CUtensorMap o0, const __grid_constant__ CUtensorMap o1,
                const __grid_constant__ GemmArgs g) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kMaxRing], s_empty[kMaxRing], s_tfull[2], s_tempty[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_dead;
    __shared__ int s_loads;  // the producer's

    constexpr bool kAMn = LAY != LAY_KK, kBMn = LAY == LAY_MM;
    constexpr bool kSums = EPI == EPI_LINEAR && (sizeof(O) == 4 || LONG);  // add sums of kStep k-blocks
    constexpr int kStep = kSums ? kChunk : 1 << 28;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = (smem_u32(smem_raw) + 1023) & ~1023u;
    // CG 2: a pair of CTAs (rank 0 and 1 of a cluster) works on 256 features; each loads its 128 and half
    // of the tokens, rank 0 issues the products for both, and either holds its own rows' sums.
    const int own = g.bn / CG;  // tokens that this CTA loads
    const int bbytes = own * kBK * 2, sbytes = kABytes + bbytes;
    const uint32_t full = smem_u32(s_full), empty = smem_u32(s_empty);
    const uint32_t tfull = smem_u32(s_tfull), tempty = smem_u32(s_tempty), drain = smem_u32(&s_drain);
    uint32_t cols = 32;
    while ((int)cols < 2 * g.bn) cols *= 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < g.stages; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(tfull + 8 * i, 1), mbar_init(tempty + 8 * i, 8 * CG);
        mbar_init(drain, 1);
        s_dead = 0;
        fence_barrier_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch(&a0);
        tma_prefetch(&b0);
    }
    if (warp == 9) tmem_alloc<CG>(smem_u32(&s_tmem), cols);
    tc_fence_before();
    if constexpr (CG == 2) cluster_sync_all();  // the barriers of both are there
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const Guard dead{&s_dead, g.waits};
    // What came before on the stream may still run until here; the next launch may start its own
    // set-up as this one's CTAs end.
    if (!g.beside) grid_wait();
    grid_release();

    const int member = CG == 2 ? (int)cluster_rank() : 0;  // of the pair
    const int rank = CG == 1 && g.splits > 1 ? (int)cluster_rank() : 0;
    const int team = CG == 2 ? 2 : g.splits;  // CTAs of a tile
    const int first = blockIdx.x / team, step = gridDim.x / team;
    const int tiles = g.n_tiles * g.t_tiles;
    const int k_lo = (int)((long long)g.kb * rank / g.splits), k_hi = (int)((long long)g.kb * (rank + 1) / g.splits);

    // Tile order: kGroup token tiles together, weight tiles advancing: the CTAs at work at one
    // time then share a few token tiles and a few weight tiles, which L2 serves.
    auto place = [&](int tile, int& tn, int& tt) {  // true: a tile of the second product
        const int per = kGroup * g.n_tiles, grp = tile / per, in = tile % per;
        const int size = min(kGroup, g.t_tiles - grp * kGroup);
        tn = in / size;
        tt = grp * kGroup + in % size;
        if constexpr (CG == 2) tn = 2 * tn + member;
        const bool second = kBMn && g.t_half > 0 && tt >= g.t_half;
        if (second) tt -= g.t_half;
        return second;
    };

    auto give_up = [&]() {  // tells the other CTA of a pair
        if constexpr (CG == 2) st_cluster_u32(map_rank(smem_u32(const_cast<int*>(&s_dead)), member ^ 1), 1);
    };

    if (warp >= 8) {
      set_regs_down<kAuxRegs>();
      // The two roles run in one thread each, and at a few hundred clocks per k-block it is their
      // instructions that bound the kernel: ring position, phase and descriptors are carried
      // along, not computed from a count, and the next barrier is looked at ahead of its use.
      const int stages = g.stages, bn = g.bn;
      const uint32_t to_empty = empty - full;
      if (warp == 8) {  // ---------------------------------------------- producer
        if (elect_one()) {
            int st = 0, loads = 0;
            uint32_t ph = 1, bar = full, at = ring;
            bool ok = true, ready = true;  // the ring starts empty
            for (int tile = first; tile < tiles && ok; tile += step) {
                int tn, tt;
                const bool second = place(tile, tn, tt);
                const int an = tn * (EPI == EPI_LINEAR ? 128 : 64), bt = tt * bn + member * own;
                int kb = k_lo;
#pragma unroll
                for (int seg = 0; seg < 2; ++seg) {  // the first operand pair, the second
                    const int end = seg ? k_hi : min(g.kb0, k_hi);
                    const CUtensorMap *ma = seg ? &a1 : &a0, *mb = seg || second ? &b1 : &b0;
                    int k = (kb - (seg ? g.kb0 : 0)) * kBK;
#pragma unroll 1
                    for (; kb < end && ok; ++kb, k += kBK) {
                        if (!ready && !(ok = mbar_wait(bar + to_empty, ph, dead))) break;
                        const uint32_t here = CG == 2 ? map_rank(bar, 0) : bar, sa = at, sb = at + kABytes;
                        const uint32_t bar_now = bar;
                        at += sbytes, bar += 8;
                        if (++st == stages) st = 0, ph ^= 1, at = ring, bar = full;
                        ready = mbar_test(bar + to_empty, ph);
                        if (member == 0) mbar_expect(bar_now, CG * sbytes);
                        if constexpr (EPI != EPI_LINEAR) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                tma_2d<CG>(sa + q * 4096, &a0, k, an + q * 16, here);
                                tma_2d<CG>(sa + q * 4096 + 2048, &a1, k, an + q * 16, here);
                            }
                        } else if constexpr (kAMn) {
                            tma_2d<CG>(sa, ma, an, k, here);
                            tma_2d<CG>(sa + kABytes / 2, ma, an + 64, k, here);
                        } else {
                            tma_2d<CG>(sa, ma, k, an, here);
                        }
                        if constexpr (kBMn) {
                            for (int j = 0; j < own; j += 64) tma_2d<CG>(sb + j * 128, mb, bt + j, k, here);
                        } else {
                            tma_2d<CG>(sb, mb, k, bt, here);
                        }
                        ++loads;
                    }
                }
            }
            if (ok && CG == 2)  // the pair's arrivals on this CTA's barriers
                for (int i = loads > stages ? loads - stages : 0; i < loads && ok; ++i)
                    ok = mbar_wait(empty + 8 * (i % stages), (i / stages) & 1, dead);
            s_loads = loads;
            if (!ok) give_up();
        }
        __syncwarp();
      } else if (warp == 9) {  // --------------------------------------- issuer
        if (member == 0 && elect_one()) {
            const uint64_t a_first = make_desc(ring, kAMn ? 8192 : 16, 1024);
            const uint64_t b_first = make_desc(ring + kABytes, kBMn ? 8192 : 16, 1024);
            constexpr uint32_t kAStep = kAMn ? 2048 >> 4 : 32 >> 4, kBStep = kBMn ? 2048 >> 4 : 32 >> 4;
            const uint32_t idesc = g.idesc, hop = (uint32_t)sbytes >> 4;
            int st = 0, local = 0;  // local: accumulators so far
            uint32_t ph = 0, bar = full, off = 0;
            bool ok = first >= tiles || mbar_first(full, 0, dead), ready = false;
            for (int tile = first; tile < tiles && ok; tile += step)
              for (int kb = k_lo; kb < k_hi && ok; ++local) {
                const int buf = local & 1, c_hi = min(k_hi, kb + kStep);
                if (!(ok = mbar_wait(tempty + 8 * buf, ((local >> 1) & 1) ^ 1, dead))) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * bn;
                bool add = false;
#pragma unroll 1
                for (; kb < c_hi; ++kb) {
                    if (!ready && !(ok = mbar_wait(bar, ph, dead))) break;
                    tc_fence_after();
                    const uint64_t da = a_first + off, db = b_first + off;
                    const uint32_t done = bar + to_empty;
                    off += hop, bar += 8;
                    if (++st == stages) st = 0, ph ^= 1, off = 0, bar = full;
                    ready = mbar_test(bar, ph);
#pragma unroll
                    for (int ks = 0; ks < kBK / 16; ++ks) {
                        mma_ss<CG>(d, da + ks * kAStep, db + ks * kBStep, idesc, add);
                        add = true;
                    }
                    if constexpr (CG == 2) tc_commit_pair(done);
                    else tc_commit(done);
                }
                if (ok) {
                    if constexpr (CG == 2) tc_commit_pair(tfull + 8 * buf);
                    else tc_commit(tfull + 8 * buf);
                }
            }
            if (!ok) give_up();
        }
        __syncwarp();
      }
      if (g.splits > 1) {  // the epilogue's two meetings of the cluster
          __syncwarp();
          cluster_sync_all();
          cluster_sync_all();
      }
    } else {  // ------------------------------------------------------ epilogue
        set_regs_up<kEpiRegs>();
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        Out w{&o0, &o1, smem_raw + (ring - smem_u32(smem_raw)) + kRingBytes + warp * kStageBytes, 0, quad, lane};
        auto give_back = [&](uint32_t bar) {  // to the issuer, of the pair's first CTA
            if constexpr (CG == 2) mbar_arrive_cluster(map_rank(bar, 0));
            else mbar_arrive(bar);
        };
        int local = 0;
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step) {
            int tn, tt;
            const bool second = place(tile, tn, tt);
            float bias = 0.f;
            if constexpr (EPI == EPI_LINEAR) {
                const int64_t n = (int64_t)tn * 128 + quad * 32 + lane;
                if (g.bias && n < g.N) bias = to_f<T>(((const T*)g.bias)[n]);
            }
            const int64_t t0 = (int64_t)tt * g.bn;
            const int valid = (int)min((int64_t)g.bn, g.M - t0);
            // columns of this warp: blocks of 32 (16 in the narrowest tile), every other one
            auto finish = [&](int c, const float* v) {
                if (g.splits > 1) {  // the partial tile, [token][feature], for the cluster to sum
                    float* part = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)));
                    const int n = g.bn >= 32 ? 32 : 16;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < n) part[(c + j) * 128 + quad * 32 + lane] = v[j];
                } else if (g.bn >= 32) {
                    emit_act<EPI, LAY, 32, T, O>(g, w, v, tn, t0 + c, bias, second);
                } else {
                    emit_act<EPI, LAY, 16, T, O>(g, w, v, tn, t0 + c, bias, second);
                }
            };
            auto fetch = [&](uint32_t src, uint32_t* r) {
                if (g.bn >= 32) tmem_ld32(src, r);
                else tmem_ld16(src, r);
                tmem_wait_ld();
            };
            if constexpr (kSums) {
                float acc[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[i][j] = 0.f;
                for (int c_lo = k_lo; c_lo < k_hi && ok; c_lo += kStep, ++local) {
                    const int buf = local & 1;
                    if (!(ok = mbar_wait_all(tfull + 8 * buf, (local >> 1) & 1, dead))) break;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = half * 32 + 64 * i;
                        if (c >= valid) break;
                        uint32_t r[32];
                        fetch(tmem + buf * g.bn + lanes + c, r);
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[i][j] += __uint_as_float(r[j]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) give_back(tempty + 8 * buf);
                }
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = half * 32 + 64 * i;
                    if (c >= valid) break;
                    finish(c, acc[i]);
                }
            } else {
                const int buf = local & 1;
                if (!(ok = mbar_wait_all(tfull + 8 * buf, (local >> 1) & 1, dead))) break;
                tc_fence_after();
                for (int c = half * 32; c < valid; c += 64) {
                    uint32_t r[32];
                    fetch(tmem + buf * g.bn + lanes + c, r);
                    finish(c, reinterpret_cast<const float*>(r));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) give_back(tempty + 8 * buf);
                ++local;
            }
        }
        if (!ok && lane == 0) give_up();
        if (g.splits > 1) {
            __syncwarp();
            cluster_sync_all();
            if (!s_dead) {
                int tn, tt;
                const bool second = place(first, tn, tt);
                const int64_t t0 = (int64_t)tt * g.bn;
                const int valid = (int)min((int64_t)g.bn, g.M - t0);
                const int pairs = (valid + 1) / 2;
                // Every CTA's share of a pair of columns is asked for before the first is used.
                auto join = [&](auto count) {
                    constexpr int S = decltype(count)::value;
                    // two pairs at a time, with what the epilogue adds to them
                    for (int u0 = rank * 8 + warp; u0 < 4 * pairs; u0 += 16 * S) {
                        float part[2][S][2], add[2][2], bias[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int u = min(u0 + i * 8 * S, 4 * pairs - 1), quad = u & 3, c = (u >> 2) * 2;
                            bias[i] = add[i][0] = add[i][1] = 0.f;
                            if constexpr (EPI == EPI_LINEAR) {
                                const int64_t n = (int64_t)tn * 128 + quad * 32 + lane;
                                if (g.bias && n < g.N) bias[i] = to_f<T>(((const T*)g.bias)[n]);
                                if (g.res && n < g.N) {
                                    const O* res = (const O*)g.res + (t0 + c) * g.ld_res + n;
                                    add[i][0] = to_f<O>(res[0]);
                                    if (c + 1 < valid) add[i][1] = to_f<O>(res[g.ld_res]);
                                }
                            }
                            const uint32_t at = ring + (uint32_t)(c * 128 + quad * 32 + lane) * 4;
#pragma unroll
                            for (int s = 0; s < S; ++s) {
                                const uint32_t ra = map_rank(at, s);
                                part[i][s][0] = ld_cluster_f32(ra);
                                part[i][s][1] = ld_cluster_f32(ra + 512);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int u = u0 + i * 8 * S;
                            if (u >= 4 * pairs) break;
                            float v[2] = {part[i][0][0], part[i][0][1]};
#pragma unroll
                            for (int s = 1; s < S; ++s) v[0] += part[i][s][0], v[1] += part[i][s][1];
                            w.quad = u & 3;
                            emit_act<EPI, LAY, 2, T, O>(g, w, v, tn, t0 + (u >> 2) * 2, bias[i], second, add[i]);
                        }
                    }
                };
                if (g.splits == 2) join(std::integral_constant<int, 2>{});
                else if (g.splits == 4) join(std::integral_constant<int, 4>{});
                else join(std::integral_constant<int, 8>{});
            }
            __syncwarp();
            cluster_sync_all();
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the stage has been read
        __syncwarp();
    }
    if (g.beside) grid_wait();
    tc_fence_before();
    if constexpr (CG == 2) {
        __syncwarp();
        cluster_sync_all();  // neither leaves while the other reads its memory or arrives on its barriers
    } else {
        __syncthreads();
    }
    tc_fence_after();
    if (__builtin_expect(s_dead, 0)) {
        if (warp == 9 && elect_one()) unwind_products<CG>(member == 0, drain);
        if (warp == 8 && elect_one()) unwind_loads<CG>(full, g.stages, s_loads);
        __syncwarp();
        if constexpr (CG == 2) cluster_sync_all();
        else __syncthreads();
    }
    if (warp == 9) tmem_free<CG>(tmem, cols);
}

// ------------------------------------------------------------------ a few tokens
// One to four tokens against weights whose rows run over k: a warp takes a row (the gated block: the
// gate and the up row of a feature) or, when rows are few, two, four or eight warps share it; each
// lane reads 16 bytes at a time and adds in fp32; the tokens' rows come from L1. Bound by the weights' bytes; the tensor-core kernel above takes as long
// at the memory's rate, but its start, its ring and its split cost two or three microseconds more,
// which is half of a small call: see few_tokens().
struct RowArgs {
    const void *x, *w0, *w1, *bias, *res;
    void* out;
    int64_t ld_x, ld_w0, ld_w1, ld_res, ld_out, n;
    int k, m, act;
    int share;  // warps of a row
};
constexpr int kRowThreads = 256;
constexpr int kRowBatch = 6;                       // 16-byte reads of a row under way (4 of two rows)
constexpr int kRowShare = 8;                       // warps of a row, at most
constexpr int kRowHop = 16384;                     // elements, not less than a step over k
static_assert(256 * kRowShare * kRowBatch <= kRowHop, "a step over k");

// Eight values in one register quad (a load of its own: the compiler would else load them one by one).
template <typename T>
__device__ __forceinline__ void widen(const uint4& v, float* f) {
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) Half2<T>::unpack(q[i], f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ uint4 ld_kept(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_stream(const void* p) {  // read once: not kept in L1
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float act_any(int act, float z) {
    switch (act) {
        case KD_ACT_RELU: return act_fn<KD_ACT_RELU>(z);
        case KD_ACT_SILU: return act_fn<KD_ACT_SILU>(z);
        case KD_ACT_GELU: return act_fn<KD_ACT_GELU>(z);
        default: return z;
    }
}

template <int M, bool GATED, typename T, typename O>
__global__ void __launch_bounds__(kRowThreads) row_kernel(const __grid_constant__ RowArgs g) {
    constexpr int R = GATED ? 2 : 1, kBatch = GATED ? 4 : kRowBatch;  // rows of a warp, reads of a row under way
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31;
    __shared__ float s_sum[kRowThreads / 32][R][M];
    const int warp = threadIdx.x >> 5, part = warp % g.share;
    const int64_t n = ((int64_t)blockIdx.x * (kRowThreads / 32) + warp) / g.share;
    const bool live = n < g.n;
    const int64_t row = live ? n : g.n - 1;
    const T* w[R];
    w[0] = (const T*)g.w0 + row * g.ld_w0;
    if constexpr (GATED) w[1] = (const T*)g.w1 + row * g.ld_w1;
    const T* x = (const T*)g.x;
    float acc[R][M];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < M; ++t) acc[r][t] = 0.f;
    const int whole = g.k & ~7;
    const int hop = 256 * g.share;
    for (int k0 = (part * 32 + lane) * 8; k0 < whole; k0 += hop * kBatch) {
        uint4 v[kBatch][R];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int r = 0; r < R; ++r)
                v[b][r] = k0 + hop * b < whole ? ld_stream(w[r] + k0 + hop * b) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int k = k0 + hop * b;
            if (k >= whole) break;
            float a[R][8];
#pragma unroll
            for (int r = 0; r < R; ++r) widen<T>(v[b][r], a[r]);
#pragma unroll
            for (int t = 0; t < M; ++t) {
                if (t >= g.m) break;
                float f[8];
                widen<T>(ld_kept(x + t * g.ld_x + k), f);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[r][t] = fmaf(a[r][i], f[i], acc[r][t]);
            }
        }
    }
    if (part == 0 && whole + lane < g.k) {  // the last elements of a k that is no multiple of 8
#pragma unroll
        for (int t = 0; t < M; ++t)
            if (t < g.m)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    acc[r][t] = fmaf(to_f<T>(w[r][whole + lane]), to_f<T>(x[t * g.ld_x + whole + lane]), acc[r][t]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < M; ++t)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
    if (g.share > 1) {  // a row's first warp adds up, in the order of the warps
        if (lane == 0)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < M; ++t) s_sum[warp][r][t] = acc[r][t];
        __syncthreads();
        if (part != 0) return;
        for (int p = 1; p < g.share; ++p)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < M; ++t) acc[r][t] += s_sum[warp + p][r][t];
    }
    if (!live) return;
#pragma unroll
    for (int t = 0; t < M; ++t) {  // lane t writes token t
        if (lane != t || t >= g.m) continue;
        O* out = (O*)g.out + t * g.ld_out + n;
        if constexpr (GATED) {
            *out = from_f<O>(act_any(g.act, acc[0][t]) * acc[R - 1][t]);
        } else {
            const float b = g.bias ? to_f<T>(((const T*)g.bias)[n]) : 0.f;
            const float r = g.res ? to_f<O>(((const O*)g.res)[t * g.ld_res + n]) : 0.f;
            *out = from_f<O>(act_any(g.act, acc[0][t] + b) + r);
        }
    }
}

template <bool GATED, typename T, typename O>
int run_rows(RowArgs g, cudaStream_t stream) {
    // sixteen warps for every SM, as long as a warp of a row still reads its batch
    int sms = 0;
    if (int rc = op_sm_count(&sms)) return rc;
    g.share = 1;
    while (g.share < kRowShare && g.n * g.share < sms * 16 && g.k >= 256 * 2 * g.share) g.share *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((g.n * g.share + kRowThreads / 32 - 1) / (kRowThreads / 32)));
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (g.m == 1) e = cudaLaunchKernelEx(&cfg, row_kernel<1, GATED, T, O>, g);
    else if (g.m == 2) e = cudaLaunchKernelEx(&cfg, row_kernel<2, GATED, T, O>, g);
    else e = cudaLaunchKernelEx(&cfg, row_kernel<4, GATED, T, O>, g);
    if (e != cudaSuccess) return op_fail(KD_ECUDA, "launch failed: %s", cudaGetErrorString(e));
    return KD_OK;
}

// Whether the row kernel is the quicker one (rows: weight matrices, 1 or 2). One token: at every size
// measured (us in graphs, row kernel and tensor cores: 64 x 64 1.7 / 3.8, 1,536 x 1,536 3.1 / 5.2, 4,096 x 4,096
// 9.6 / 10.5, 128,256 x 4,096 151 / 160). A further token costs it a read and eight products for every 16
// bytes of weights, and the tensor cores nothing: two tokens 2,048 x 2,048 4.6 / 5.6, 1,536 x 4,096 6.8 /
// 6.1; four 1,536 x 1,536 5.2 / 5.4, 2,048 x 2,048 6.0 / 5.7.
bool few_tokens(int64_t m, int64_t n, int64_t k, int rows) {
    return m == 1 || (m <= 4 && (double)m * n * k * rows <= 9.5e6);
}

// ------------------------------------------------------------------ launch
struct Operand {
    const void* p;
    int64_t ld;  // elements between rows
    bool mn;     // rows run over k (the M or N index is the contiguous one)
};

// Tile width (tokens) and split of the reduction, by an estimate of the time in microseconds.
// A k-block costs an SM what its instructions or its product take (measured from one-tile
// runs: 0.20 us up to 64 columns, 0.28 at 128, 0.41 at 256, about linear between), or the CTAs' loads at
// 10.5 TB/s, whichever is more (fitted to the widths that turned out best; that it is L2's rate is not shown:
// pairs of CTAs load a quarter less of the gated block of 128 x 2,048 x 8,192, which takes 19 us either way); a
// tile's epilogue runs beside the next tile's products; a split costs its exchange. Both sides, measured (us):
// 128 x 4,096 x 2,048: 32 columns 14.1, 128 columns split by four 15.5; 128 x 1,536 x 4,096: 16
// columns 17.8, 128 split by eight 11.2; 1,024 x 2,048 x 2,048: 128 columns 13.6, 256 19.4.
struct Plan {
    int bn, splits, grid;
};

// room[s]: clusters of s CTAs that the device runs at once (a GPU processing cluster holds whole ones:
// fewer than sms / s; 128 CTAs in clusters of eight take two rounds).
// Widths are multiples of 32 (of 64 where the tokens are the contiguous index of B), so that 257
// tokens, say, are two tiles of 160 (257 x 6,290 x 9,142: 72 us, as three of 128 or two of 256 101).
Plan make_plan(int64_t n_tiles, int64_t M, int kb, int sms, const int* room, bool b_mn) {
    Plan best{};
    double best_cost = 1e300;
    for (int bn = b_mn ? 64 : 16; bn <= 256; bn = bn < 32 ? 32 : bn + (b_mn ? 64 : 32)) {
        const int64_t tiles = n_tiles * ((M + bn - 1) / bn);
        for (int s = 1; s <= 8; s *= 2) {
            if (s > 1 && (2 * s > kb || tiles > room[s])) break;
            const double work = bn <= 64 ? 0.20 + bn * 0.0003 : 0.155 + bn * 0.001;
            const double ctas = (double)(tiles * s < sms ? tiles * s : sms);
            const double load = ctas * (kABytes + 128.0 * bn) / 10.5e6;
            const double body = (double)((kb + s - 1) / s) * (work > load ? work : load), tail = 0.4 + 0.012 * bn;
            const double waves = (double)((tiles * s + sms - 1) / sms);
            const double cost = s > 1 ? body + tail / s + 2.0 + 0.025 * bn : waves * (body > tail ? body : tail) + tail;
            if (cost < best_cost) {
                best_cost = cost;
                best.bn = bn;
                best.splits = s;
                best.grid = (int)(s > 1 ? tiles * s : (tiles < sms ? tiles : sms));
            }
        }
        if (bn >= M) break;
    }
    return best;
}

template <int CG, int EPI, int LAY, typename T, typename O, bool LONG = false>
int launch(const CUtensorMap* m, const GemmArgs& g, int grid, cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    static std::atomic<bool> ready[64];
    if (dev >= 64 || !ready[dev].load()) {
        cudaError_t e = cudaFuncSetAttribute(gemm_kernel<CG, EPI, LAY, T, O, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSmemBytes);
        if (e != cudaSuccess) return op_fail(KD_ECUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        if (dev < 64) ready[dev].store(true);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CG == 2 ? 2 : g.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CG == 2 || g.splits > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, gemm_kernel<CG, EPI, LAY, T, O, LONG>, m[0], m[1], m[2], m[3], m[4], m[5], g);
    if (e != cudaSuccess) return op_fail(KD_ECUDA, "launch failed: %s", cudaGetErrorString(e));
    return KD_OK;
}

int cluster_room(int sms, int room[9]) {
    static std::atomic<int> cached[64][3];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return op_fail(KD_ECUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    for (int i = 0, s = 2; s <= 8; ++i, s *= 2) {
        int n = dev < 64 ? cached[dev][i].load() : 0;
        if (n == 0) {
            const auto kernel = gemm_kernel<1, EPI_LINEAR, LAY_KK, __nv_bfloat16, __nv_bfloat16, false>;
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(sms / s * s);
            cfg.blockDim = dim3(kGemmThreads);
            cfg.dynamicSmemBytes = kSmemBytes;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = s;
            at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            if (e != cudaSuccess) return op_fail(KD_ECUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
            if (n < 1) n = -1;  // none: not asked again
            if (dev < 64) cached[dev][i].store(n);
        }
        room[s] = n;
    }
    return KD_OK;
}

int operand_map(CUtensorMap* m, int dtype, const Operand& o, int64_t rows, int64_t k, int box_rows) {
    if (o.mn) return make_map_2d(m, dtype, o.p, rows, k, o.ld, 64, kBK);
    return make_map_2d(m, dtype, o.p, k, rows, o.ld, kBK, box_rows);
}

template <int EPI, typename T, typename O>
int run_typed(GemmArgs g, int dtype, const Operand* a, const Operand* b, int pairs, int64_t k, cudaStream_t stream) {
    const bool both = pairs < 0;  // two products of a[0], with b[0] into out and b[1] into out2
    if (both) pairs = 1;
    int sms = 0;
    int room[9];
    int rc = op_sm_count(&sms);
    if (rc == KD_OK) rc = cluster_room(sms, room);
    if (rc) return rc;
    const bool gated = EPI != EPI_LINEAR;
    const int per = gated ? 64 : 128;
    const int64_t n_tiles = (g.N + per - 1) / per;
    const int64_t kblocks = (k + kBK - 1) / kBK;
    const Plan p = make_plan(both ? 2 * n_tiles : n_tiles, g.M, (int)kblocks * (gated ? 1 : pairs), sms, room, b[0].mn);
    g.kb0 = (int)kblocks;
    g.kb = (int)kblocks * (gated ? 1 : pairs);
    int64_t t_tiles = (g.M + p.bn - 1) / p.bn;
    if (both) g.t_half = (int)t_tiles, t_tiles *= 2;
    if (n_tiles * t_tiles > 0x3fffffff) return op_fail(KD_EINVAL, "too many output tiles");
    // Pairs of CTAs where they take no more rounds than single ones.
    const int64_t pair_tiles = (n_tiles + 1) / 2 * t_tiles;
    const bool pieces = EPI == EPI_LINEAR && sizeof(O) == 2 && g.kb / p.splits > (dtype == KD_BF16 ? kLongBF16 : kLongF16);
    const bool pair = !pieces && p.splits == 1 && p.bn >= kPairMin && p.bn % (b[0].mn ? 128 : 64) == 0 && n_tiles > 1 && room[2] >= sms / 2 &&
                      (pair_tiles + sms / 2 - 1) / (sms / 2) <= (n_tiles * t_tiles + sms - 1) / sms;
    const int cg = pair ? 2 : 1;
    const int grid = pair ? 2 * (int)(pair_tiles < sms / 2 ? pair_tiles : sms / 2) : p.grid;
    g.n_tiles = (int)(pair ? (n_tiles + 1) / 2 : n_tiles);
    g.t_tiles = (int)t_tiles;
    g.bn = p.bn;
    g.splits = p.splits;
    g.stages = kRingBytes / (kABytes + p.bn / cg * kBK * 2);
    if (g.stages > kMaxRing) g.stages = kMaxRing;
    g.idesc = make_idesc(128 * cg, p.bn, dtype == KD_BF16, a[0].mn, b[0].mn);
    CUtensorMap m[6];  // A, A of the second pair, B, the second B, the outputs
    const int a_box = gated ? 16 : 128;
    if ((rc = operand_map(&m[0], dtype, a[0], g.N, k, a_box))) return rc;
    if ((rc = operand_map(&m[2], dtype, b[0], g.M, k, p.bn / cg))) return rc;
    m[1] = m[0];
    m[3] = m[2];
    if (pairs > 1 && (rc = operand_map(&m[1], dtype, a[1], g.N, k, a_box))) return rc;
    if ((both || (pairs > 1 && !gated)) && (rc = operand_map(&m[3], dtype, b[1], g.M, k, p.bn / cg))) return rc;
    const bool two = both || EPI == EPI_GATED_BWD;
    const int out_type = sizeof(O) == 4 ? KD_F32 : dtype;
    if (!two) g.ld_out2 = g.ld_out, g.out2 = g.out;
    if (EPI == EPI_GATED_BWD) g.ld_out2 = g.ld_out;
    int64_t ld[2] = {g.ld_out, g.ld_out2};
    const void* out[2] = {g.out, g.out2};
    g.tma_out = 1;
    for (int i = 0; i < 2; ++i) {
        if (g.M == 1) ld[i] = (g.N + 7) & ~(int64_t)7;  // one row: its distance to the next is not used
        if ((uintptr_t)out[i] % 16 || ld[i] * (int64_t)sizeof(O) % 16 || ld[i] >= (int64_t)1 << 37) g.tma_out = 0;
    }
    m[4] = m[5] = m[0];
    if (g.tma_out && p.splits == 1) {
        const int rows = sizeof(O) == 4 || p.bn < 32 ? 16 : 32;
        if ((rc = make_map_out(&m[4], out_type, out[0], g.N, g.M, ld[0], gated ? 16 : 32, rows))) return rc;
        if (two && (rc = make_map_out(&m[5], out_type, out[1], g.N, g.M, ld[1], gated ? 16 : 32, rows))) return rc;
    }
    if constexpr (EPI == EPI_LINEAR) {
        if constexpr (sizeof(O) == 2)
            if (pieces)
                return b[0].mn   ? launch<1, EPI, LAY_MM, T, O, true>(m, g, grid, stream)
                       : a[0].mn ? launch<1, EPI, LAY_MK, T, O, true>(m, g, grid, stream)
                                 : launch<1, EPI, LAY_KK, T, O, true>(m, g, grid, stream);
        if constexpr (sizeof(O) == 2)  // the weights' gradients
            if (b[0].mn) return pair ? launch<2, EPI, LAY_MM, T, O>(m, g, grid, stream) : launch<1, EPI, LAY_MM, T, O>(m, g, grid, stream);
        if (a[0].mn) return pair ? launch<2, EPI, LAY_MK, T, O>(m, g, grid, stream) : launch<1, EPI, LAY_MK, T, O>(m, g, grid, stream);
    }
    return pair ? launch<2, EPI, LAY_KK, T, O>(m, g, grid, stream) : launch<1, EPI, LAY_KK, T, O>(m, g, grid, stream);
}

template <int EPI>
int run(const GemmArgs& g, int dtype, int out_dtype, const Operand* a, const Operand* b, int pairs, int64_t k,
        cudaStream_t s) {
    if constexpr (EPI == EPI_LINEAR) {
        if (out_dtype == KD_F32)
            return dtype == KD_BF16 ? run_typed<EPI, __nv_bfloat16, float>(g, dtype, a, b, pairs, k, s)
                                    : run_typed<EPI, __half, float>(g, dtype, a, b, pairs, k, s);
    }
    return dtype == KD_BF16 ? run_typed<EPI, __nv_bfloat16, __nv_bfloat16>(g, dtype, a, b, pairs, k, s)
                            : run_typed<EPI, __half, __half>(g, dtype, a, b, pairs, k, s);
}

bool known_act(int a) { return a >= KD_ACT_NONE && a <= KD_ACT_GELU; }

// A 16-bit matrix that TMA reads: 16-byte aligned base, and rows that start on 16 bytes.
int check_operand(const char* what, const void* p, int64_t rows, int64_t cols, int64_t* ld) {
    if (!p) return op_fail(KD_EINVAL, "%s: NULL pointer", what);
    if ((uintptr_t)p & 15) return op_fail(KD_EINVAL, "%s: not 16-byte aligned", what);
    if (rows == 1) {  // the distance of rows is not used
        *ld = (cols + 7) & ~(int64_t)7;
        return KD_OK;
    }
    if (*ld < cols || *ld % 8 || *ld >= (int64_t)1 << 38)
        return op_fail(KD_EINVAL, "%s: rows of %lld elements, %lld apart (need a multiple of 8, at least the row)", what,
                       (long long)cols, (long long)*ld);
    return KD_OK;
}

int check_rows(const char* what, const void* p, int elem, int64_t rows, int64_t cols, int64_t ld) {
    if (!p) return op_fail(KD_EINVAL, "%s: NULL pointer", what);
    if ((uintptr_t)p % elem) return op_fail(KD_EINVAL, "%s: misaligned pointer", what);
    if (rows > 1 && ld < cols) return op_fail(KD_EINVAL, "%s: rows of %lld elements, %lld apart", what, (long long)cols, (long long)ld);
    return KD_OK;
}

// TMA coordinates are 32-bit, and so is the row kernel's k, which steps past the end by less than a hop.
constexpr int64_t kMaxDim = ((int64_t)1 << 31) - kRowHop;

int check_sizes(const char* who, int dtype, int act, int64_t m, int64_t n, int64_t k) {
    if (dtype != KD_BF16 && dtype != KD_F16) return op_fail(KD_EINVAL, "%s: dtype must be KD_BF16 or KD_F16", who);
    if (!known_act(act)) return op_fail(KD_EINVAL, "%s: unknown activation %d", who, act);
    if (m < 0 || n < 0 || k < 1 || m > kMaxDim || n > kMaxDim || k > kMaxDim)
        return op_fail(KD_EINVAL, "%s: sizes m=%lld n=%lld k=%lld out of range", who, (long long)m, (long long)n, (long long)k);
    return KD_OK;
}

}  // namespace

int gemm_status(cudaStream_t s, unsigned int* st) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(st, g_op_status, sizeof *st, 0, cudaMemcpyDeviceToHost, s);
    const unsigned int zero = 0;
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *st) {
        e = cudaMemcpyToSymbolAsync(g_op_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e == cudaSuccess ? KD_OK : op_fail(KD_ECUDA, "kd_op_sync: %s", cudaGetErrorString(e));
}

int linear_op(const kd_linear_args* p, const OpWaits& waits, cudaStream_t s) {
    if (!p) return op_fail(KD_EINVAL, "kd_linear: NULL arguments");
    kd_linear_args q = *p;
    int rc = check_sizes("kd_linear", q.dtype, q.act, q.m, q.n, q.k);
    if (rc) return rc;
    if (q.out_dtype != q.dtype && q.out_dtype != KD_F32)
        return op_fail(KD_EINVAL, "kd_linear: out_dtype must be the input type or KD_F32");
    if (q.w_transposed != 0 && q.w_transposed != 1) return op_fail(KD_EINVAL, "kd_linear: w_transposed must be 0 or 1");
    if (q.m == 0 || q.n == 0) return KD_OK;
    const int oe = q.out_dtype == KD_F32 ? 4 : 2;
    if ((rc = check_operand("kd_linear: x", q.x, q.m, q.k, &q.ld_x))) return rc;
    if ((rc = check_operand("kd_linear: w", q.w, q.w_transposed ? q.k : q.n, q.w_transposed ? q.n : q.k, &q.ld_w))) return rc;
    if (q.bias && (uintptr_t)q.bias % 2) return op_fail(KD_EINVAL, "kd_linear: bias: misaligned pointer");
    if (q.residual && (rc = check_rows("kd_linear: residual", q.residual, oe, q.m, q.n, q.ld_residual))) return rc;
    if ((rc = check_rows("kd_linear: out", q.out, oe, q.m, q.n, q.ld_out))) return rc;
    if (few_tokens(q.m, q.n, q.k, 1) && !q.w_transposed) {
        const RowArgs r{q.x, q.w, nullptr, q.bias, q.residual, q.out, q.ld_x, q.ld_w, 0, q.ld_residual, q.ld_out, q.n, (int)q.k, (int)q.m, q.act};
        if (q.dtype == KD_BF16)
            return q.out_dtype == KD_F32 ? run_rows<false, __nv_bfloat16, float>(r, s) : run_rows<false, __nv_bfloat16, __nv_bfloat16>(r, s);
        return q.out_dtype == KD_F32 ? run_rows<false, __half, float>(r, s) : run_rows<false, __half, __half>(r, s);
    }
    GemmArgs g{};
    g.N = q.n, g.M = q.m, g.act = q.act, g.waits = waits;
    g.bias = q.bias, g.res = q.residual, g.ld_res = q.ld_residual, g.out = q.out, g.ld_out = q.ld_out;
    const Operand a{q.w, q.ld_w, q.w_transposed != 0}, b{q.x, q.ld_x, false};
    return run<EPI_LINEAR>(g, q.dtype, q.out_dtype, &a, &b, 1, q.k, s);
}

static int check_gated(const char* who, kd_gated_args* q) {
    int rc = check_sizes(who, q->dtype, q->act, q->m, q->f, q->d);
    if (rc) return rc;
    if (q->m == 0 || q->f == 0) return KD_OK;
    if ((rc = check_operand("gated block: x", q->x, q->m, q->d, &q->ld_x))) return rc;
    if ((rc = check_operand("gated block: wg", q->wg, q->f, q->d, &q->ld_wg))) return rc;
    return check_operand("gated block: wu", q->wu, q->f, q->d, &q->ld_wu);
}

int gated_op(const kd_gated_args* p, void* h, int64_t ld_h, const OpWaits& waits, cudaStream_t s) {
    if (!p) return op_fail(KD_EINVAL, "kd_gated_ffn: NULL arguments");
    kd_gated_args q = *p;
    int rc = check_gated("kd_gated_ffn", &q);
    if (rc || q.m == 0 || q.f == 0) return rc;
    if ((rc = check_rows("kd_gated_ffn: h", h, 2, q.m, q.f, ld_h))) return rc;
    if (few_tokens(q.m, q.f, q.d, 2)) {
        const RowArgs r{q.x, q.wg, q.wu, nullptr, nullptr, h, q.ld_x, q.ld_wg, q.ld_wu, 0, ld_h, q.f, (int)q.d, (int)q.m, q.act};
        return q.dtype == KD_BF16 ? run_rows<true, __nv_bfloat16, __nv_bfloat16>(r, s)
                                  : run_rows<true, __half, __half>(r, s);
    }
    GemmArgs g{};
    g.N = q.f, g.M = q.m, g.act = q.act, g.out = h, g.ld_out = ld_h, g.waits = waits;
    const Operand a[2] = {{q.wg, q.ld_wg, false}, {q.wu, q.ld_wu, false}}, b{q.x, q.ld_x, false};
    return run<EPI_GATED>(g, q.dtype, q.dtype, a, &b, 2, q.d, s);
}

}  // namespace kd

using namespace kd;

extern "C" {

const char* kd_op_error(void) { return t_err; }

int kd_op_set_timeout(int64_t ns) {
    if (ns < 1) return op_fail(KD_EINVAL, "kd_op_set_timeout: the limit must be at least 1 ns");
    t_limit_ns = ns;
    return KD_OK;
}

int kd_op_sync(void* stream) {
    unsigned int a = 0, b = 0;
    int rc = gemm_status((cudaStream_t)stream, &a);
    if (rc == KD_OK) rc = attention_status((cudaStream_t)stream, &b);
    if (rc) return rc;
    if (a | b) return op_fail(KD_ETIMEOUT, "a device-side wait of an operator exceeded its limit");
    return KD_OK;
}

int kd_linear(const kd_linear_args* p, void* stream) { return linear_op(p, own_waits(), (cudaStream_t)stream); }

int kd_gated_ffn(const kd_gated_args* p, void* h, int64_t ld_h, void* stream) {
    return gated_op(p, h, ld_h, own_waits(), (cudaStream_t)stream);
}

static int64_t gated_ld(int64_t f) { return (f + 63) & ~(int64_t)63; }

size_t kd_gated_ffn_backward_workspace(int64_t m, int64_t f) {
    if (m < 0 || f < 0 || m > kMaxDim || f > kMaxDim) return 0;
    return (size_t)m * gated_ld(f) * 2 * 2 + 256;
}

int kd_gated_ffn_backward(const kd_gated_args* p, const void* dh, int64_t ld_dh, void* dx, int64_t ld_dx, void* dwg,
                          int64_t ld_dwg, void* dwu, int64_t ld_dwu, void* workspace, size_t workspace_bytes,
                          void* stream) {
    if (!p) return op_fail(KD_EINVAL, "kd_gated_ffn_backward: NULL arguments");
    kd_gated_args q = *p;
    int rc = check_gated("kd_gated_ffn_backward", &q);
    if (rc) return rc;
    if (q.m == 0 || q.f == 0) return op_fail(KD_EINVAL, "kd_gated_ffn_backward: m and f must be at least 1");
    if ((rc = check_rows("kd_gated_ffn_backward: dh", dh, 2, q.m, q.f, ld_dh))) return rc;
    if (dx && (rc = check_rows("kd_gated_ffn_backward: dx", dx, 2, q.m, q.d, ld_dx))) return rc;
    if (dwg && (rc = check_rows("kd_gated_ffn_backward: dwg", dwg, 2, q.f, q.d, ld_dwg))) return rc;
    if (dwu && (rc = check_rows("kd_gated_ffn_backward: dwu", dwu, 2, q.f, q.d, ld_dwu))) return rc;
    if (!workspace || workspace_bytes < kd_gated_ffn_backward_workspace(q.m, q.f))
        return op_fail(KD_ENOMEM, "kd_gated_ffn_backward: workspace of %zu bytes, need %zu", workspace_bytes,
                       kd_gated_ffn_backward_workspace(q.m, q.f));
    const int64_t ld = gated_ld(q.f);
    uint8_t* base = (uint8_t*)(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    uint8_t* dg = base;
    uint8_t* du = base + (size_t)q.m * ld * 2;
    cudaStream_t s = (cudaStream_t)stream;
    // dg = dh u act'(g), du = dh act(g), with g and u recomputed. They are rounded to the input
    // type once: the next two products take 16-bit operands, and one more rounding of the terms
    // of a sum is of the size of the rounding of its result.
    {
        GemmArgs g{};
        g.waits = own_waits();
        g.N = q.f, g.M = q.m, g.act = q.act, g.res = dh, g.ld_res = ld_dh, g.out = dg, g.out2 = du, g.ld_out = ld;
        const Operand a[2] = {{q.wg, q.ld_wg, false}, {q.wu, q.ld_wu, false}}, b{q.x, q.ld_x, false};
        if ((rc = run<EPI_GATED_BWD>(g, q.dtype, q.dtype, a, &b, 2, q.d, s))) return rc;
    }
    if (dx) {  // dx[t][c] = sum_f dg[t][f] wg[f][c] + du[t][f] wu[f][c]: one sum over both pairs
        GemmArgs g{};
        g.waits = own_waits();
        g.N = q.d, g.M = q.m, g.out = dx, g.ld_out = ld_dx;
        const Operand a[2] = {{q.wg, q.ld_wg, true}, {q.wu, q.ld_wu, true}}, b[2] = {{dg, ld, false}, {du, ld, false}};
        if ((rc = run<EPI_LINEAR>(g, q.dtype, q.dtype, a, b, 2, q.f, s))) return rc;
    }
    // dwg[f][c] = sum_t dg[t][f] x[t][c], dwu from du: one launch for both
    const Operand a{q.x, q.ld_x, true}, b[2] = {{dwg ? dg : du, ld, true}, {du, ld, true}};
    if (dwg || dwu) {
        GemmArgs g{};
        g.waits = own_waits();
        g.N = q.d, g.M = q.f;
        g.out = dwg ? dwg : dwu, g.ld_out = dwg ? ld_dwg : ld_dwu;
        g.out2 = dwu, g.ld_out2 = ld_dwu;
        g.beside = dx != nullptr;
        if ((rc = run<EPI_LINEAR>(g, q.dtype, q.dtype, &a, b, dwg && dwu ? -1 : 1, q.m, s))) return rc;
    }
    return KD_OK;
}

}  // extern "C"
