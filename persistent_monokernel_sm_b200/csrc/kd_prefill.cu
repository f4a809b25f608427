// kd_prefill.cu -- a prompt through the decoder at once: kd_prefill runs the layers over all its
// tokens but the last with the operators of kd_gemm.cu and kd_attention.cu, straight from the
// arena's streaming layout (the Q/K/V rows as they lie, gate and up rows as two matrices of
// stride 2 d, the output and down projections as the transposed matrices they are), and leaves
// the last token pending for kd_decode. The kernels here are the steps between the products:
// embedding + RMSNorm, RMSNorm, and RoPE with the cache append. They move a few megabytes per
// layer of a 128-token prompt (nothing beside the weights); each is one pass, a block per token.
//
// Precision: the residual, the Q/K/V outputs, norms and RoPE are fp32; what the tensor cores
// take as an operand (normalised activations, q, attention outputs, hidden units) is rounded to
// bf16 once, and k and v once, when they are appended, as in kd_decode.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kd.h"
#include "kd_layout.h"
#include "kd_ops.h"

using namespace kd;

int kd_internal_view(kd_ctx* ctx, kd_ctx_view* v);
int kd_internal_fail(kd_ctx* ctx, int code, const char* msg);
void kd_internal_count_launch(kd_ctx* ctx);

namespace {

constexpr int kNormThreads = 256;

// xn[t] = bf16(x[t] / rms(x[t]) * gain), one block per token; with `embed`, x[t] is first
// gathered from the embedding row of tokens[t]. A token id outside the vocabulary sets the
// handle's status (kd_sync reports KD_ETOKEN) and its row is taken as zero.
__global__ void __launch_bounds__(kNormThreads)
    norm_rows(float* x, __nv_bfloat16* xn, const __nv_bfloat16* gain, int d, float eps, const __nv_bfloat16* embed,
              const int32_t* tokens, int vocab, unsigned long long* ctl) {
    __shared__ float part[kNormThreads / 32];
    const int64_t t = blockIdx.x;
    float* row = x + t * d;
    float v[kMaxModel / kNormThreads];
    constexpr int kVec = kMaxModel / kNormThreads / 4;
    int id = 0;
    bool in = true;
    if (embed) {
        id = tokens[t];
        in = id >= 0 && id < vocab;
        if (!in && threadIdx.x == 0 && atomicCAS(ctl + kCtlStatus, 0ull, (unsigned long long)kStatusToken) == 0ull)
            ctl[kCtlWhere] = (unsigned long long)(t & 0xff);
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = (i * kNormThreads + threadIdx.x) * 4;
        if (c < d) {
            if (embed) {
                const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(embed + (int64_t)(in ? id : 0) * d + c);
                const float2 a = __bfloat1622float2(e[0]), b = __bfloat1622float2(e[1]);
                v[4 * i] = in ? a.x : 0.f, v[4 * i + 1] = in ? a.y : 0.f;
                v[4 * i + 2] = in ? b.x : 0.f, v[4 * i + 3] = in ? b.y : 0.f;
                *reinterpret_cast<float4*>(row + c) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else {
                const float4 a = *reinterpret_cast<const float4*>(row + c);
                v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sum = fmaf(v[4 * i + j], v[4 * i + j], sum);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) sum += part[i];
    const float r = 1.f / sqrtf(sum / (float)d + eps);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = (i * kNormThreads + threadIdx.x) * 4;
        if (c < d) {
            const __nv_bfloat162* g = reinterpret_cast<const __nv_bfloat162*>(gain + c);
            const float2 a = __bfloat1622float2(g[0]), b = __bfloat1622float2(g[1]);
            __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(xn + t * d + c);
            o[0] = __floats2bfloat162_rn(v[4 * i] * r * a.x, v[4 * i + 1] * r * a.y);
            o[1] = __floats2bfloat162_rn(v[4 * i + 2] * r * b.x, v[4 * i + 3] * r * b.y);
        }
    }
}

// One block per token: rotates the pairs of q and k (adjacent outputs of the arena's Q/K/V rows
// are dims i and i + hd/2) by the token's row of the (cos, sin) table, writes q [t][Hq][hd] and
// appends k and v to the cache at position pos0 + t.
__global__ void __launch_bounds__(256)
    rope_append(const float* qkv, const float2* table, __nv_bfloat16* q, __nv_bfloat16* kc, __nv_bfloat16* vc, Dims dm,
                int pos0) {
    const int64_t t = blockIdx.x, pos = pos0 + t;
    const int half = dm.hd / 2, per = (dm.r + 2) * half;
    const float2* in = reinterpret_cast<const float2*>(qkv + t * dm.qkv_rows);
    const float2* cs = table + pos * half;
    for (int p = threadIdx.x; p < dm.Hkv * per; p += blockDim.x) {
        const int g = p / per, rest = p % per, head = rest / half, i = rest % half;
        const float2 v = in[p];
        if (head == dm.r + 1) {
            __nv_bfloat16* o = vc + ((int64_t)g * dm.S + pos) * dm.hd + 2 * i;
            *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(v.x, v.y);
        } else {
            const float2 r = cs[i];
            __nv_bfloat16* o = head < dm.r ? q + (t * dm.Hq + g * dm.r + head) * dm.hd
                                           : kc + ((int64_t)g * dm.S + pos) * dm.hd;
            o[i] = __float2bfloat16_rn(v.x * r.x - v.y * r.y);
            o[i + half] = __float2bfloat16_rn(v.y * r.x + v.x * r.y);
        }
    }
}

// The workspace of c tokens: the residual, and one region that holds in turn the Q/K/V outputs
// and q, then the hidden units; normalised activations and attention outputs share another.
struct Space {
    size_t x, xn, qkv, q, att, h, part, total;
};
size_t up(size_t v) { return (v + 255) & ~(size_t)255; }
int64_t hidden_ld(int F) { return (F + 7) & ~7; }

Space space_of(const Dims& d, int64_t c) {
    Space s;
    s.x = 0;
    s.xn = up((size_t)c * d.d * 4);
    s.att = s.xn;  // the normalised activations are used up by the Q/K/V product
    const size_t a = (size_t)c * d.d * 2, b = (size_t)c * d.qd * 2;
    s.qkv = s.xn + up(a > b ? a : b);
    s.q = s.qkv + up((size_t)c * d.qkv_rows * 4);
    const size_t qkv_q = s.q + up((size_t)c * d.qd * 2) - s.qkv;
    s.h = s.qkv;
    const size_t h = up((size_t)c * hidden_ld(d.F) * 2);
    s.part = s.qkv + (qkv_q > h ? qkv_q : h);
    // attention's partial results, whatever the size of a piece (the last may be small)
    s.total = s.part + kAttnPartBytes;
    return s;
}

}  // namespace

namespace kd {
bool dims_of(const kd_config* cfg, Dims* d);  // kd_api.cu: false for an invalid configuration
}

extern "C" {

size_t kd_prefill_workspace(const kd_config* cfg, int32_t n_tokens) {
    Dims d;
    if (!dims_of(cfg, &d) || n_tokens < 1) return 0;
    return space_of(d, n_tokens).total + 256;
}

int kd_prefill(kd_ctx* c, const int32_t* d_tokens, int32_t n_tokens, int32_t kv_len, void* workspace,
               size_t workspace_bytes) {
    kd_ctx_view v;
    if (!c || kd_internal_view(c, &v) != KD_OK) return KD_EINVAL;
    const Dims& d = *v.dm;
    const Layout& y = *v.lay;
    if (!v.has_weights) return kd_internal_fail(c, KD_ESTATE, "kd_prefill: no weights loaded");
    if (!d_tokens || n_tokens < 1 || kv_len < 0) return kd_internal_fail(c, KD_EINVAL, "kd_prefill: bad tokens or kv_len");
    if ((int64_t)kv_len + n_tokens > d.S) return kd_internal_fail(c, KD_ECAPACITY, "kd_prefill: kv_len + n_tokens exceeds max_seq");
    const int64_t n = n_tokens - 1;
    uint8_t* base = (uint8_t*)(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    const size_t lost = base - (uint8_t*)workspace;
    const size_t room = workspace && workspace_bytes > lost ? workspace_bytes - lost : 0;
    int64_t chunk = n;  // tokens taken at once: all that the workspace holds
    if (n > 0 && space_of(d, chunk).total > room) {
        int64_t lo = 0, hi = n;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            (space_of(d, mid).total <= room ? lo : hi) = mid;
        }
        chunk = lo;
        if (chunk < 1) return kd_internal_fail(c, KD_ENOMEM, "kd_prefill: the workspace does not hold one token");
    }
    // The last token is pending at its position; the cache before it is filled below.
    int rc = kd_reset(c, d_tokens + n, 1, (int32_t)(kv_len + n));
    if (rc || n == 0) return rc;

    cudaStream_t s = (cudaStream_t)v.stream;
    const Space sp = space_of(d, chunk);
    float* x = (float*)(base + sp.x);
    __nv_bfloat16 *xn = (__nv_bfloat16*)(base + sp.xn), *q = (__nv_bfloat16*)(base + sp.q);
    __nv_bfloat16 *att = (__nv_bfloat16*)(base + sp.att), *h = (__nv_bfloat16*)(base + sp.h);
    float* qkv = (float*)(base + sp.qkv);
    const int64_t ldh = hidden_ld(d.F);
    unsigned long long* ctl = (unsigned long long*)(v.arena + y.ctl);
    const OpWaits waits{op_clocks(v.timeout_ns), ctl};
    auto op = [&](int code) {
        if (code == KD_OK) kd_internal_count_launch(c);
        else kd_internal_fail(c, code, kd_op_error());
        return code;
    };
    auto own = [&]() {
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return kd_internal_fail(c, KD_ECUDA, cudaGetErrorString(e));
        kd_internal_count_launch(c);
        return (int)KD_OK;
    };
    for (int64_t at = 0; at < n; at += chunk) {
        const int64_t m = n - at < chunk ? n - at : chunk;
        const int pos0 = (int)(kv_len + at);
        for (int l = 0; l < d.L; ++l) {
            const uint8_t* w = v.arena + y.layer0 + (size_t)l * y.layer_stride;
            const size_t layer_kv = (size_t)l * d.Hkv * d.S * d.hd * 2;
            __nv_bfloat16* kc = (__nv_bfloat16*)(v.arena + y.kcache + layer_kv);
            __nv_bfloat16* vc = (__nv_bfloat16*)(v.arena + y.vcache + layer_kv);
            norm_rows<<<(unsigned)m, kNormThreads, 0, s>>>(
                x, xn, (const __nv_bfloat16*)(w + y.l_attn_norm), d.d, d.eps,
                l == 0 ? (const __nv_bfloat16*)(v.arena + y.embed) : nullptr, d_tokens + at, d.V, ctl);
            if ((rc = own())) return rc;
            kd_linear_args a{};
            a.dtype = KD_BF16, a.out_dtype = KD_F32;
            a.m = m, a.n = d.qkv_rows, a.k = d.d;
            a.x = xn, a.ld_x = d.d, a.w = w + y.l_wqkv, a.ld_w = d.d, a.out = qkv, a.ld_out = d.qkv_rows;
            if ((rc = op(linear_op(&a, waits, s)))) return rc;
            rope_append<<<(unsigned)m, 256, 0, s>>>(qkv, (const float2*)(v.arena + y.rope), q, kc, vc, d, pos0);
            if ((rc = own())) return rc;
            if (l == d.L - 1) break;  // nothing later reads what the last layer does with these tokens
            kd_attention_args t{};
            t.dtype = KD_BF16, t.n_heads = d.Hq, t.n_kv_heads = d.Hkv, t.head_dim = d.hd;
            t.n = m, t.kv_len = pos0;
            t.q = q, t.q_token = d.qd, t.q_head = d.hd;
            t.k = kc, t.v = vc, t.k_pos = t.v_pos = d.hd, t.k_head = t.v_head = (int64_t)d.S * d.hd;
            t.out = att, t.out_token = d.qd, t.out_head = d.hd;
            t.scale = 1.f / sqrtf((float)d.hd);
            t.workspace = base + sp.part, t.workspace_bytes = sp.total - sp.part;
            if ((rc = op(attention_op(&t, waits, s)))) return rc;
            if (kd_prompt_attention_workspace(&t) > 0) kd_internal_count_launch(c);  // and its join
            a = kd_linear_args{};  // x += att wo^T
            a.dtype = KD_BF16, a.out_dtype = KD_F32, a.w_transposed = 1;
            a.m = m, a.n = d.d, a.k = d.qd;
            a.x = att, a.ld_x = d.qd, a.w = w + y.l_wot, a.ld_w = d.d;
            a.residual = x, a.ld_residual = d.d, a.out = x, a.ld_out = d.d;
            if ((rc = op(linear_op(&a, waits, s)))) return rc;
            norm_rows<<<(unsigned)m, kNormThreads, 0, s>>>(x, xn, (const __nv_bfloat16*)(w + y.l_ffn_norm), d.d, d.eps,
                                                          nullptr, nullptr, 0, nullptr);
            if ((rc = own())) return rc;
            kd_gated_args f{};
            f.dtype = KD_BF16, f.act = KD_ACT_SILU;
            f.m = m, f.d = d.d, f.f = d.F;
            f.x = xn, f.ld_x = d.d;
            f.wg = w + y.l_wgu, f.wu = w + y.l_wgu + (size_t)d.d * 2, f.ld_wg = f.ld_wu = 2 * (int64_t)d.d;
            if ((rc = op(gated_op(&f, h, ldh, waits, s)))) return rc;
            a.k = d.F;  // x += h wd^T
            a.x = h, a.ld_x = ldh, a.w = w + y.l_wdt;
            if ((rc = op(linear_op(&a, waits, s)))) return rc;
        }
    }
    return KD_OK;
}

}  // extern "C"
