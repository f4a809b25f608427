// kd_attention.cu -- causal attention of n new tokens over a key-value cache that holds kv_len
// earlier positions and the new ones, on the 5th-generation tensor cores.
//
// o_i = sum_j p_ij v_j, p_i = softmax_j(scale q_i . k_j) over the positions j <= kv_len + i; in
// one pass over j with a running maximum m, sum l and unnormalised output o (online softmax).
//
// Rows: the r query heads of a kv head share its keys and values, so a tile's 128 rows are
// 128 / r tokens x r heads: keys and values are read once per kv head, and one token of a
// grouped model is one tile. A thread owns a row: no reduction crosses threads.
//
// A CTA has two streams, each a warpgroup with its own scores (128 x 128 fp32) and output
// (128 x hd fp32) in tensor memory; while one does its softmax the tensor cores work for the
// other. For prompts the streams are two neighbouring tiles that share every key and value
// block. With few tiles they share one tile and take alternate blocks, and the blocks are
// split over several CTAs besides: the partial (m, l, o) of the streams are joined in shared
// memory, those of the CTAs through a workspace by join_kernel, in a fixed order.
//
// Per block and stream: S = Q K^T; p = 2^(s - m) in 16 bits written over S; O += P V with P
// read from tensor memory. A row's reference m is raised (and O rescaled) only when its maximum
// has grown by more than 2^8: p then stays within 2^8 and O within range of fp32.
// p is rounded to 16 bits as an operand of the second product (off by half a step of its type,
// averaged over the row); its sum l is taken in fp32 before that rounding.
//
// What bounds it: for prompts the chain softmax -> P V -> next Q K^T of a stream, 2,900 clocks a
// pair of blocks where the products alone take 2,048 and the exponentials 2,048 (4,096 tokens, 32/8
// heads of 128: 124 to 136 us in a graph of eight calls, by the box, 1.0 to 1.1 PFLOP/s; 142 to 145 in
// a loop of seconds, under the power cap). At head dim 128 the softmax spills 48 bytes a thread. A
// polynomial for a part of the exponentials made it longer (2/8 of them: 130 -> 137 us): the FMA pipe has
// no room either; so did two threads a row (121 -> 139 us): the exponentials' unit is what a stream's
// softmax takes. One token: HBM and a fixed 8 us of start, last block and join (32,768 positions, 16/8
// heads: 31 us where L2 holds a part of the cache, 37 over three caches in turn, 3.6 TB/s; 131,072: 88 us,
// 6.1 TB/s).
//
// The one pass with a running maximum and sum is the online softmax of Milakov and Gimelshein (2018,
// arXiv 1805.02867). The tensor cores truncate O's sum towards zero, 9.8e-8 relative for every 16
// positions where the values have one sign: half a step of fp16 at 80,000 positions of a stream (4,096
// tokens behind 131,072: 8.6e-4 low), of bf16 at 640,000.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "kd.h"
#include "kd_ops.h"
#include "kd_sm100.h"

namespace kd {
namespace {

// Two warpgroups of softmax and one with the producer's and the issuer's warp, which gives the
// others registers: 256 x 216 + 128 x 72 = 384 x 168, the launch's total.
constexpr int kThr = 384;
constexpr int kRowRegs = 216, kAuxRegs = 72;
constexpr int kKeys = 128;  // positions per block
constexpr float kLazy = 8.f;

struct AttnArgs {
    int n, kv_len, r, hkv;
    int tq;      // tokens per tile
    int tiles;   // query tiles
    int splits;  // CTAs that share the blocks of a tile (and of a kv head)
    float* parts;  // their partial outputs: [CTA][row][HD outputs, m, l, 2 unused]
    int shared;  // the streams share a tile (alternate blocks)
    uint32_t idesc_s, idesc_o;
    float scale_log2;
    void* out;
    int64_t out_token, out_head;
    OpWaits waits;
};

template <int HD> struct Shape {
    static constexpr int block = kKeys * HD * 2;           // bytes of a key, value or query tile
    static constexpr int slots = HD == 128 ? 5 : 8;        // of the ring of key and value blocks
    static constexpr int part = HD + 4;                    // floats between rows of a partial output
    static constexpr int smem = 1024 + (2 + slots) * block;
    static_assert(2 * 128 * part * 4 <= slots * block, "the partial outputs fit the ring");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in a 64-bit register, and Blackwell's packed arithmetic on them.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo2(f2 v) {
    return __uint_as_float((uint32_t)v);
}
__device__ __forceinline__ float hi2(f2 v) {
    return __uint_as_float((uint32_t)(v >> 32));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }

// HD / 32 neighbouring outputs of a row, from one lane.
template <int HD, typename T>
__device__ __forceinline__ void store_row(const AttnArgs& a, int tok, int head, int lane, const float* o, float inv) {
    constexpr int E = HD / 32;
    T* out = (T*)a.out + (int64_t)tok * a.out_token + (int64_t)head * a.out_head + lane * E;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) w[e / 2] = Half2<T>::pack(o[e] * inv, o[e + 1] * inv);
    if constexpr (E == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(out) = w[0];
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15};" ::KD_I8(r, 0),
        KD_I8(r, 8), "r"(addr)
        : "memory");
}

template <int HD, typename T>
__global__ void __launch_bounds__(kThr, 1)
    attention_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnArgs a) {
    constexpr int kSlots = Shape<HD>::slots, kBlock = Shape<HD>::block, kPart = Shape<HD>::part, kHalves = HD / 64;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kSlots], s_empty[kSlots], s_q, s_s[2], s_p[4], s_o[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_dead;
    __shared__ int s_loads;  // the producer's, of the ring

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t qs = (smem_u32(smem_raw) + 1023) & ~1023u;
    const uint32_t ring = qs + 2 * kBlock;
    const uint32_t full = smem_u32(s_full), empty = smem_u32(s_empty), qbar = smem_u32(&s_q);
    const uint32_t sbar = smem_u32(s_s), pbar = smem_u32(s_p), obar = smem_u32(s_o), drain = smem_u32(&s_drain);
    const Guard dead{&s_dead, a.waits};
    // (m, l) of the two streams' rows for the join: where a second query tile would be
    float* stat = reinterpret_cast<float*>(smem_raw + (qs + kBlock - smem_u32(smem_raw)));
    auto part_at = [&](int s, int row) {  // a row's partial output, where the blocks were
        return reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw))) + (s * 128 + row) * kPart;
    };

    // What this CTA works on: a kv head, one or two tiles, a range of blocks per stream.
    const int rank = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
    const int g = unit % a.hkv;
    int tile[2], nb[2], lo = 0, total;  // nb: blocks of each stream; total: blocks streamed
    auto blocks_of = [&](int t) {
        const int last = min(a.n, (t + 1) * a.tq);  // one past its last token
        return (a.kv_len + last + kKeys - 1) / kKeys;
    };
    if (a.shared) {
        tile[0] = tile[1] = a.tiles - 1 - unit / a.hkv;
        const int all = blocks_of(tile[0]);
        lo = (int)((long long)all * rank / a.splits);
        total = (int)((long long)all * (rank + 1) / a.splits) - lo;
        nb[0] = (total + 1) / 2, nb[1] = total / 2;
    } else {  // the longest rows first
        const int pair = (a.tiles + 1) / 2 - 1 - unit / a.hkv;
        tile[0] = 2 * pair, tile[1] = 2 * pair + 1;
        nb[0] = blocks_of(tile[0]);
        nb[1] = tile[1] < a.tiles ? blocks_of(tile[1]) : 0;
        total = max(nb[0], nb[1]);
    }
    // Order of the ring: K_0 (and K_1 with alternate blocks), then V_i, K_(i + ahead) in turn;
    // the issuer uses them in this order.
    const int ahead = min(a.shared ? 2 : 1, total);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
        mbar_init(qbar, 1);
        for (int i = 0; i < 2; ++i) mbar_init(sbar + 8 * i, 1), mbar_init(pbar + 16 * i, 4), mbar_init(pbar + 16 * i + 8, 4), mbar_init(obar + 8 * i, 1);
        mbar_init(drain, 1);
        s_dead = 0;
        fence_barrier_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
    }
    if (warp == 9) tmem_alloc(smem_u32(&s_tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_wait();
    // Not before a join: its CTAs would wait on the few SMs that are free now and run there alone.
    if (a.splits == 1) grid_release();
    const uint32_t tmem = s_tmem;  // columns: S0, S1 (128 each), O0, O1 (HD each)

    if (warp >= 8) {
      set_regs_down<kAuxRegs>();
      if (warp == 8) {  // ---------------------------------------------- producer
        if (elect_one()) {
            const int two = !a.shared && tile[1] < a.tiles ? 2 : 1;
            mbar_expect(qbar, two * kHalves * a.tq * a.r * 128);
            for (int s = 0; s < two; ++s)
                for (int h = 0; h < kHalves; ++h)
                    tma_3d(qs + s * kBlock + h * 16384, &mq, h * 64, g * a.r, tile[s] * a.tq, qbar);
            int st = 0, loads = 0;
            uint32_t ph = 1;
            bool ok = true;
            auto load = [&](const CUtensorMap* m, int block) {
                if (!ok || !(ok = mbar_wait(empty + 8 * st, ph, dead))) return;
                mbar_expect(full + 8 * st, kBlock);
#pragma unroll
                for (int h = 0; h < kHalves; ++h)
                    tma_3d(ring + st * kBlock + h * 16384, m, h * 64, (lo + block) * kKeys, g, full + 8 * st);
                ++loads;
                if (++st == kSlots) st = 0, ph ^= 1;
            };
            for (int i = 0; i < ahead; ++i) load(&mk, i);
            for (int i = 0; i < total && ok; ++i) {
                load(&mv, i);
                if (i + ahead < total) load(&mk, i + ahead);
            }
            s_loads = loads;
        }
        __syncwarp();
    } else if (warp == 9) {  // --------------------------------------- issuer
        if (elect_one()) {
            // This thread has to keep ahead of two streams' softmax: slots and descriptors are
            // carried along, and the blocks of an iteration are waited for before its weights.
            constexpr uint32_t kHop = kBlock >> 4;
            const uint64_t q_desc = make_desc(qs, 16, 1024), k_desc = make_desc(ring, 16, 1024);
            const uint64_t v_desc = make_desc(ring, 16384, 1024);
            const uint32_t idesc_s = a.idesc_s, idesc_o = a.idesc_o;
            const int n0 = nb[0], n1 = nb[1];
            int slot = 0;
            uint32_t ph = 0;
            bool ok = mbar_first(qbar, 0, dead) && mbar_wait(qbar, 0, dead);
            auto take = [&]() {  // the next slot of the ring, once it is filled
                const int at = slot;
                ok = ok && mbar_wait(full + 8 * at, ph, dead);
                if (++slot == kSlots) slot = 0, ph ^= 1;
                return at;
            };
            auto scores = [&](int s, int at) {  // S_s = Q K^T
                const uint64_t kd = k_desc + (uint32_t)at * kHop, qd = q_desc + (a.shared ? 0u : (uint32_t)s * kHop);
#pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks) {
                    const uint32_t off = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                    mma_ss(tmem + s * 128, qd + off, kd + off, idesc_s, ks > 0);
                }
                tc_commit(sbar + 8 * s);
            };
            auto values = [&](int s, int i, int at, bool last) {  // O_s += P_s V; i: block of the stream
                const uint64_t vd = v_desc + (uint32_t)at * kHop;
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // as the weights of three quarters, of all are there
                    if (!(ok = ok && mbar_wait(pbar + 16 * s + 8 * part, i & 1, dead))) return;
                    tc_fence_after();
#pragma unroll
                    for (int ks = 6 * part; ks < 6 + 2 * part; ++ks)
                        mma_ts(tmem + 256 + s * HD, tmem + s * 128 + ks * 8, vd + ks * (2048 >> 4), idesc_o, i > 0 || ks > 0);
                }
                if (last) tc_commit(obar + 8 * s);
            };
            if (a.shared) {
                for (int i = 0; i < ahead && ok; ++i) {
                    const int k = take();
                    if (!ok) break;
                    tc_fence_after();
                    scores(i, k);
                    tc_commit(empty + 8 * k);
                }
                for (int i = 0; i < total && ok; ++i) {
                    const int s = i & 1, v = take(), k = i + 2 < total ? take() : -1;
                    if (!ok) break;
                    values(s, i >> 1, v, i + 2 >= total);
                    if (!ok) break;
                    if (k >= 0) scores(s, k);
                    tc_commit(empty + 8 * v);
                    if (k >= 0) tc_commit(empty + 8 * k);
                }
            } else {
                const int first = take();
                if (ok) {
                    tc_fence_after();
                    scores(0, first);
                    if (n1 > 0) scores(1, first);
                    tc_commit(empty + 8 * first);
                }
                for (int i = 0; i < total && ok; ++i) {
                    const int v = take(), k = i + 1 < total ? take() : -1;
                    if (!ok) break;
                    if (i < n0) {
                        values(0, i, v, i == n0 - 1);
                        if (!ok) break;
                        if (i + 1 < n0) scores(0, k);
                    }
                    if (i < n1) {
                        values(1, i, v, i == n1 - 1);
                        if (!ok) break;
                        if (i + 1 < n1) scores(1, k);
                    }
                    tc_commit(empty + 8 * v);
                    if (k >= 0) tc_commit(empty + 8 * k);
                }
            }
        }
        __syncwarp();
      }
      if (a.shared) __syncthreads();  // the streams' join
    } else {  // ------------------------------------------------------ softmax
        set_regs_up<kRowRegs>();
        const int s = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t at = (uint32_t)(quad * 32) << 16;
        const uint32_t S = tmem + s * 128 + at, O = tmem + 256 + s * HD + at;
        const int tok = tile[s] * a.tq + row / a.r;
        const bool live = row < a.tq * a.r && tok < a.n;
        const bool any = __any_sync(0xffffffffu, live);  // else the warp only keeps the barriers going
        const int seen = a.kv_len + tok + 1;             // positions this row sees
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < nb[s]; ++i) {
            if (!(ok = mbar_wait_all(sbar + 8 * s, i & 1, dead))) break;
            if (any) {
                tc_fence_after();
                uint32_t z[kKeys];
                const int left = seen - (lo + (a.shared ? 2 * i + s : i)) * kKeys;  // keys of this block it sees
                const bool cut = __any_sync(0xffffffffu, left < kKeys);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                tmem_ld32(S, z);
                tmem_ld32(S + 32, z + 32);
                tmem_wait_ld();
                tmem_ld32(S + 64, z + 64);
                tmem_ld32(S + 96, z + 96);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (half) tmem_wait_ld();
                    if (cut) {
#pragma unroll
                        for (int c = 64 * half; c < 64 * half + 64; ++c)
                            if (c >= left) z[c] = 0xff800000u;
                    }
#pragma unroll
                    for (int c = 64 * half; c < 64 * half + 64; c += 2)
                        mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(z[c]), __uint_as_float(z[c + 1]));
                }
                const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * a.scale_log2;
                // m is the reference in log2 units; -inf while the row has seen nothing
                const bool grow = top > m + kLazy || (m == -INFINITY && top > -INFINITY);
                if (__any_sync(0xffffffffu, grow)) {
                    const float to = grow ? top : m;
                    const float f = m == -INFINITY ? 0.f : ex2(m - to);
                    l *= f;
                    m = to;
                    if (i > 0) {
#pragma unroll
                        for (int c = 0; c < HD; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(O + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st32(O + c, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : -m;
                const f2 scale2 = both(a.scale_log2), ref2 = both(ref);
                f2 sum[2] = {0ull, 0ull};
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // three quarters, then the last
#pragma unroll
                    for (int c = 96 * part; c < 96 + 32 * part; c += 32) {
                        uint32_t p[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const f2 x = fma2(pack2(__uint_as_float(z[c + 2 * j]), __uint_as_float(z[c + 2 * j + 1])), scale2, ref2);
                            const f2 e = pack2(ex2(lo2(x)), ex2(hi2(x)));
                            sum[j & 1] = add2(sum[j & 1], e);
                            p[j] = Half2<T>::pack(lo2(e), hi2(e));
                        }
                        tmem_st16(S + c / 2, p);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(pbar + 16 * s + 8 * part);
                }
                const f2 all = add2(sum[0], sum[1]);
                l += lo2(all) + hi2(all);
            } else if (lane == 0) {
                mbar_arrive(pbar + 16 * s);
                mbar_arrive(pbar + 16 * s + 8);
            }
        }
        if (ok && nb[s] > 0) ok = mbar_wait_all(obar + 8 * s, 0, dead);
        // the partial outputs go where the blocks were: the other stream has to be done too
        if (ok && a.shared && nb[s ^ 1] > 0) ok = mbar_wait_all(obar + 8 * (s ^ 1), 0, dead);
        tc_fence_after();
        if (!a.shared) {
            if (ok && any && nb[s] > 0) {
                const float inv = 1.f / l;
                T* out = (T*)a.out + (int64_t)tok * a.out_token + (int64_t)(g * a.r + row % a.r) * a.out_head;
#pragma unroll
                for (int c = 0; c < HD; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(O + c, o);
                    tmem_wait_ld();
                    if (live) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = Half2<T>::pack(__uint_as_float(o[j + 2 * e]) * inv, __uint_as_float(o[j + 2 * e + 1]) * inv);
                            *reinterpret_cast<uint4*>(out + c + j) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
        } else {  // leave (m, l, o) for the join below; the ring is free: every copy has been used
            stat[s * 256 + row] = m;
            stat[s * 256 + 128 + row] = l;
            if (ok && any && nb[s] > 0) {
                float* part = part_at(s, row);
#pragma unroll
                for (int c = 0; c < HD; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(O + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) *reinterpret_cast<uint4*>(part + c + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
            }
        }
        tc_fence_before();
        if (a.shared) {
            // The two streams' partials of a row are joined by a warp, whose lanes hold HD / 32
            // neighbouring outputs each; a split tile's go to the workspace for join_kernel.
            __syncthreads();
            if (!s_dead) {
                const int tokens = min(a.tq, a.n - tile[0] * a.tq), rows = tokens * a.r;
                constexpr int E = HD / 32;
                for (int row = warp; row < rows; row += 8) {
                    const float m0 = stat[row], m1 = stat[256 + row], l0 = stat[128 + row], l1 = stat[384 + row];
                    const float best = fmaxf(m0, m1);
                    // A stream that saw nothing has l = 0 and may have written no output. (m does not tell: the
                    // maximum passes over NaN, so that scores of NaN alone leave it at -infinity, and l at NaN.)
                    const float w0 = l0 == 0.f ? 0.f : ex2(m0 - best), w1 = l1 == 0.f ? 0.f : ex2(m1 - best);
                    float l = 0.f, o[E];
                    const float *p0 = part_at(0, row) + lane * E, *p1 = part_at(1, row) + lane * E;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[e] = 0.f;
                    if (l0 != 0.f) {
                        l = w0 * l0;
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] = w0 * p0[e];
                    }
                    if (l1 != 0.f) {
                        l += w1 * l1;
#pragma unroll
                        for (int e = 0; e < E; ++e) o[e] = fmaf(w1, p1[e], o[e]);
                    }
                    if (a.splits == 1) {
                        store_row<HD, T>(a, tile[0] * a.tq + row / a.r, g * a.r + row % a.r, lane, o, 1.f / l);
                    } else {
                        float* to = a.parts + ((int64_t)blockIdx.x * 128 + row) * kPart;
#pragma unroll
                        for (int e = 0; e < E; ++e) to[lane * E + e] = o[e];
                        if (lane == 0) to[HD] = best, to[HD + 1] = l;
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (__builtin_expect(s_dead, 0)) {
        // A wait has given up: no thread starts anything any more; products and copies under way, whichever
        // role gave up, end before the shared and the tensor memory goes.
        if (warp == 9 && elect_one()) {
            tc_commit(drain);
            mbar_drain(drain, 0);
        }
        if (warp == 8 && elect_one()) {
            mbar_drain(qbar, 0);
            for (int i = s_loads > kSlots ? s_loads - kSlots : 0; i < s_loads; ++i)
                mbar_drain(full + 8 * (i % kSlots), (i / kSlots) & 1);
        }
        __syncthreads();
    }
    if (warp == 9) tmem_free(tmem, 512);
}

// Joins the partial rows of split tiles: a warp per row, which reads eight partials at a time.
// With m the maximum over the partials that saw anything (l_p is not 0; NaN counts as seen), o = sum
// 2^(m_p - m) o_p / sum 2^(m_p - m) l_p, in the order of p.
template <int HD, typename T>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttnArgs a) {
    grid_wait();
    constexpr int E = HD / 32, kPart = Shape<HD>::part;
    const int lane = threadIdx.x & 31, per = a.tq * a.r;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int unit = (int)(w / per), row = (int)(w % per);
    const int tile = a.tiles - 1 - unit / a.hkv, g = unit % a.hkv, tok = tile * a.tq + row / a.r;
    if (unit >= a.tiles * a.hkv || tok >= a.n) return;
    const float* from = a.parts + ((int64_t)unit * a.splits * 128 + row) * kPart;
    float best = -INFINITY;
    for (int p = lane; p < a.splits; p += 32) best = fmaxf(best, from[(int64_t)p * 128 * kPart + HD]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, x));
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int p0 = 0; p0 < a.splits; p0 += 8) {
        float v[8][E], m[8], s[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const float* at = from + (int64_t)min(p0 + p, a.splits - 1) * 128 * kPart;
            m[p] = at[HD], s[p] = at[HD + 1];
#pragma unroll
            for (int e = 0; e < E; ++e) v[p][e] = at[lane * E + e];
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p0 + p >= a.splits || s[p] == 0.f) continue;
            const float wp = ex2(m[p] - best);
            l = fmaf(wp, s[p], l);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(wp, v[p][e], o[e]);
        }
    }
    store_row<HD, T>(a, tok, g * a.r + row % a.r, lane, o, 1.f / l);
}

template <int HD, typename T>
int launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const AttnArgs& a, int grid, cudaStream_t s) {
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !ready[dev].load())) {
        e = cudaFuncSetAttribute(attention_kernel<HD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<HD>::smem);
        if (e == cudaSuccess && dev < 64) ready[dev].store(true);
    }
    if (e != cudaSuccess) return op_fail(KD_ECUDA, "kd_prompt_attention: %s", cudaGetErrorString(e));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = Shape<HD>::smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attention_kernel<HD, T>, q, k, v, a);
    if (e == cudaSuccess && a.splits > 1) {
        const int64_t rows = (int64_t)a.tiles * a.hkv * a.tq * a.r;
        cfg.gridDim = dim3((unsigned)((rows + 3) / 4));
        cfg.blockDim = dim3(128);
        cfg.dynamicSmemBytes = 0;
        e = cudaLaunchKernelEx(&cfg, join_kernel<HD, T>, a);
    }
    if (e != cudaSuccess) return op_fail(KD_ECUDA, "launch failed: %s", cudaGetErrorString(e));
    return KD_OK;
}

// How the work is cut: the CTAs, whether two streams share a tile, and the split of its blocks.
// It goes by the sizes and kCtas (the SMs of a B200) alone, so that a workspace can be sized
// without a device.
constexpr int kCtas = 148;
struct Cut {
    int shared, splits;
    int64_t grid, bytes;
};
Cut cut_of(int64_t n, int64_t kv_len, int r, int hkv, int hd) {
    const int tq = 128 / r;
    const int64_t tiles = (n + tq - 1) / tq, units = tiles * hkv, pairs = (tiles + 1) / 2 * hkv;
    const int64_t blocks = (kv_len + n + kKeys - 1) / kKeys;
    Cut c{0, 1, pairs, 0};
    // Full waves of CTAs, in tiles: rows of about the same length that just miss a whole wave of
    // pairs are better off as single tiles (1,184 tokens behind 31,000, 32/8 heads: 152 pairs 786
    // us, 304 single tiles 496 us). Shorter rows among longer ones even the pairs out by themselves.
    const int64_t pair_waves = (pairs + kCtas - 1) / kCtas, unit_waves = (units + kCtas - 1) / kCtas;
    if (units <= kCtas || (kv_len >= n && pair_waves <= 4 && unit_waves < 2 * pair_waves)) {
        // One tile per CTA; few tiles' blocks go to as many CTAs as there are SMs while each of its
        // streams keeps a block, or of a short cache the CTA one (77 tokens behind 1,001, 4/2 heads of 64: by
        // four 10.8 us, by nine 9.3; one token behind 2,000, 16/8 heads: whole 16.6, by eight 9.9; one
        // behind 32,768: by eight 37, by eighteen 31). Past sixteen, a CTA keeps six blocks: the join
        // reads every share (one token behind 32,768, 8/1 heads: by 36 19 us, by 128 28).
        c.shared = 1;
        int64_t most = blocks / 6 > 16 ? blocks / 6 : 16;
        if (most > kCtas / units) most = kCtas / units;
        const int64_t worth = blocks <= 10 ? blocks : blocks / 2;
        c.splits = (int)(most < worth ? most : worth);
        if (c.splits < 1) c.splits = 1;
        c.grid = units * c.splits;
        if (c.splits > 1) c.bytes = c.grid * 128 * (hd + 4) * 4 + 256;
    }
    return c;
}

}  // namespace

int attention_status(cudaStream_t s, unsigned int* st) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(st, g_op_status, sizeof *st, 0, cudaMemcpyDeviceToHost, s);
    const unsigned int zero = 0;
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *st) {
        e = cudaMemcpyToSymbolAsync(g_op_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e == cudaSuccess ? KD_OK : op_fail(KD_ECUDA, "kd_op_sync: %s", cudaGetErrorString(e));
}

static int check_attention(const kd_attention_args& q) {
    if (q.dtype != KD_BF16 && q.dtype != KD_F16)
        return op_fail(KD_EINVAL, "kd_prompt_attention: dtype must be KD_BF16 or KD_F16");
    if (q.head_dim != 64 && q.head_dim != 128) return op_fail(KD_EINVAL, "kd_prompt_attention: head_dim must be 64 or 128");
    if (q.n_heads < 1 || q.n_kv_heads < 1 || q.n_heads % q.n_kv_heads || q.n_heads / q.n_kv_heads > 128 || q.n_kv_heads > 65535)
        return op_fail(KD_EINVAL, "kd_prompt_attention: %d query heads over %d kv heads (need a multiple, at most 128 each)",
                       q.n_heads, q.n_kv_heads);
    if (q.n < 0 || q.kv_len < 0 || q.n > (1 << 30) || q.kv_len > (1 << 30) - q.n)
        return op_fail(KD_EINVAL, "kd_prompt_attention: n=%lld kv_len=%lld out of range", (long long)q.n, (long long)q.kv_len);
    if (!(q.scale > 0.f) || !(q.scale < INFINITY)) return op_fail(KD_EINVAL, "kd_prompt_attention: scale must be finite and > 0");
    return KD_OK;
}

int attention_op(const kd_attention_args* p, const OpWaits& waits, cudaStream_t s) {
    if (!p) return op_fail(KD_EINVAL, "kd_prompt_attention: NULL arguments");
    kd_attention_args q = *p;
    int rc = check_attention(q);
    if (rc) return rc;
    if (q.n == 0) return KD_OK;
    // the stride of a dimension of one entry is not used
    if (q.n_heads == 1) q.q_head = q.out_head = q.head_dim;
    if (q.n_kv_heads == 1) q.k_head = q.v_head = q.head_dim;
    if (q.n == 1) q.q_token = q.out_token = q.head_dim;
    if (q.n + q.kv_len == 1) q.k_pos = q.v_pos = q.head_dim;
    const void* ptr[4] = {q.q, q.k, q.v, q.out};
    const int64_t st[8] = {q.q_token, q.q_head, q.k_pos, q.k_head, q.v_pos, q.v_head, q.out_token, q.out_head};
    const char* names[4] = {"q", "k", "v", "out"};
    for (int i = 0; i < 4; ++i) {
        if (!ptr[i] || ((uintptr_t)ptr[i] & 15))
            return op_fail(KD_EINVAL, "kd_prompt_attention: %s is NULL or not 16-byte aligned", names[i]);
        for (int j = 0; j < 2; ++j)
            if (st[2 * i + j] < q.head_dim || st[2 * i + j] % 8 || st[2 * i + j] >= (int64_t)1 << 38)
                return op_fail(KD_EINVAL, "kd_prompt_attention: %s: strides must be multiples of 8, at least head_dim", names[i]);
    }
    AttnArgs a{};
    a.n = (int)q.n, a.kv_len = (int)q.kv_len;
    a.hkv = q.n_kv_heads, a.r = q.n_heads / q.n_kv_heads;
    a.tq = 128 / a.r;
    a.tiles = (a.n + a.tq - 1) / a.tq;
    a.scale_log2 = q.scale * 1.4426950408889634f;
    a.out = q.out, a.out_token = q.out_token, a.out_head = q.out_head;
    const int64_t T = q.kv_len + q.n;
    const Cut c = cut_of(q.n, q.kv_len, a.r, a.hkv, q.head_dim);
    if ((int64_t)a.tiles * a.hkv > 0x3fffffff) return op_fail(KD_EINVAL, "kd_prompt_attention: too many tiles");
    if (c.bytes > 0 && (!q.workspace || q.workspace_bytes < (size_t)c.bytes))
        return op_fail(KD_ENOMEM, "kd_prompt_attention: workspace of %zu bytes, need %zu", q.workspace ? q.workspace_bytes : 0,
                       (size_t)c.bytes);
    a.shared = c.shared, a.splits = c.splits;
    a.parts = (float*)(((uintptr_t)q.workspace + 255) & ~(uintptr_t)255);
    a.waits = waits;
    const int64_t grid = c.grid;
    const bool bf = q.dtype == KD_BF16;
    CUtensorMap mq, mk, mv;
    // Rows past the last position read as zeros (not what the cache holds there): a weight of 0
    // times it is then 0.
    if ((rc = make_map_3d(&mq, q.dtype, q.q, q.head_dim, q.n_heads, q.n, q.q_head, q.q_token, 64, a.r, a.tq))) return rc;
    if ((rc = make_map_3d(&mk, q.dtype, q.k, q.head_dim, T, a.hkv, q.k_pos, q.k_head, 64, kKeys, 1))) return rc;
    if ((rc = make_map_3d(&mv, q.dtype, q.v, q.head_dim, T, a.hkv, q.v_pos, q.v_head, 64, kKeys, 1))) return rc;
    a.idesc_s = make_idesc(128, kKeys, bf, false, false);
    a.idesc_o = make_idesc(128, q.head_dim, bf, false, true);
    if (q.head_dim == 128)
        return bf ? launch<128, __nv_bfloat16>(mq, mk, mv, a, (int)grid, s) : launch<128, __half>(mq, mk, mv, a, (int)grid, s);
    return bf ? launch<64, __nv_bfloat16>(mq, mk, mv, a, (int)grid, s) : launch<64, __half>(mq, mk, mv, a, (int)grid, s);
}

}  // namespace kd

using namespace kd;

extern "C" size_t kd_prompt_attention_workspace(const kd_attention_args* p) {
    if (!p || check_attention(*p) || p->n == 0) return 0;
    return (size_t)cut_of(p->n, p->kv_len, p->n_heads / p->n_kv_heads, p->n_kv_heads, p->head_dim).bytes;
}

extern "C" int kd_prompt_attention(const kd_attention_args* p, void* stream) {
    return attention_op(p, own_waits(), (cudaStream_t)stream);
}
