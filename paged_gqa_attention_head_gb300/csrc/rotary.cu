// Query/key preparation of a layer's new tokens: an RMS norm of each head's row and the
// position rotation, in one pass over q and k.
//
//     y = x * rsqrt(mean(x^2) + eps) * w          (per head row of D; without weights y = x)
//     (y_a, y_b) -> mscale (y_a cos t - y_b sin t, y_b cos t + y_a sin t),   t = position * theta_i
//
// for pair i of the first R elements: (i, i + R/2) in the half layout, (2i, 2i + 1) in the
// interleaved one.  One rounding, of the result to bf16; sums and rotations in fp32, the
// angle within ~1e-6 rad (rope.cuh).
//
// Bound by HBM: 2 D bytes in and 2 D out per row.  A row is held by D/8 lanes, each with two
// 8-byte chunks whose pairs it can turn alone: chunks c and c + R/8 in the half layout, two
// neighbours in the interleaved one.  So a row needs no exchange beyond the norm's 3 or 4
// shuffles, and every 32-byte sector a warp touches is used whole: 16381 tokens of 72 rows of 64 take
// 51.0 us, 5.9 TB/s (with two 16-byte chunks a lane a warp held 114 registers, four blocks fitted an
// SM, and it took 67.5 us).  The angles depend on the token only: a warp works for one
// token, takes its R/2 (cos, sin) once into shared memory (one or two sincos per lane) and uses
// them for all of its rows.
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace sinkattn {
namespace {

constexpr int kRotWarps = 4;
constexpr int kRotBatch = 4;

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// What a lane's eight elements of a row are multiplied by: the firsts x and seconds y of four pairs,
// two pairs in each float2 (one instruction works on both).
struct Turn {
    float2 xc[2], ys[2], yc[2], xs[2];  // w_x cos, -w_y sin, w_y cos, w_x sin
};

// Passes p0 .. p1 - 1 over the H rows of one tensor of one token.
template <int D, bool kInterleaved>
__device__ __forceinline__ void run_rows(const __nv_bfloat16 *src, __nv_bfloat16 *dst, int H, int p0, int p1,
                                         const float *weight, float eps, const float2 (&cs)[4], bool rot, int ea,
                                         int eb, int row_in_pass) {
    constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = kRotBatch;
    if (p0 >= p1) return;  // warp-uniform
    const int row0 = p0 * kRows + row_in_pass;
    src += (int64_t)row0 * D;
    dst += (int64_t)row0 * D;
    uint2 a[kBatch], b[kBatch];
    // rows from p0 that this lane's part of the passes still has
    const int mine = min(H - row0, (p1 - p0) * kRows - row_in_pass);
    auto load = [&](int p) {  // passes p0 + p ..
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if ((p + j) * kRows < mine) {
                const __nv_bfloat16 *x = src + (p + j) * kRows * D;
                a[j] = *reinterpret_cast<const uint2 *>(x + ea);
                b[j] = *reinterpret_cast<const uint2 *>(x + eb);
            }
    };
    load(0);
    Turn t;
    {
        float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
        if (weight) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(weight + ea));
            const float4 g = __ldg(reinterpret_cast<const float4 *>(weight + eb));
            wa[0] = f.x, wa[1] = f.y, wa[2] = f.z, wa[3] = f.w;
            wb[0] = g.x, wb[1] = g.y, wb[2] = g.z, wb[3] = g.w;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 wx = kInterleaved ? (i ? make_float2(wb[0], wb[2]) : make_float2(wa[0], wa[2]))
                                           : make_float2(wa[2 * i], wa[2 * i + 1]);
            const float2 wy = kInterleaved ? (i ? make_float2(wb[1], wb[3]) : make_float2(wa[1], wa[3]))
                                           : make_float2(wb[2 * i], wb[2 * i + 1]);
            const float2 c = make_float2(cs[2 * i].x, cs[2 * i + 1].x), s = make_float2(cs[2 * i].y, cs[2 * i + 1].y);
            t.xc[i] = fmul2(wx, c);
            t.yc[i] = fmul2(wy, c);
            t.ys[i] = fmul2(wy, make_float2(-s.x, -s.y));
            t.xs[i] = fmul2(wx, s);
        }
    }
    for (int p = 0; p < p1 - p0; p += kBatch) {
        if (p > 0) load(p);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const bool ok = (p + j) * kRows < mine;
            if (!__any_sync(0xffffffffu, ok)) break;
            float2 x[2], y[2];
            if (kInterleaved) {
                x[0] = make_float2(bf_lo(a[j].x), bf_lo(a[j].y));
                y[0] = make_float2(bf_hi(a[j].x), bf_hi(a[j].y));
                x[1] = make_float2(bf_lo(b[j].x), bf_lo(b[j].y));
                y[1] = make_float2(bf_hi(b[j].x), bf_hi(b[j].y));
            } else {
                x[0] = make_float2(bf_lo(a[j].x), bf_hi(a[j].x));
                x[1] = make_float2(bf_lo(a[j].y), bf_hi(a[j].y));
                y[0] = make_float2(bf_lo(b[j].x), bf_hi(b[j].x));
                y[1] = make_float2(bf_lo(b[j].y), bf_hi(b[j].y));
            }
            float2 inv = make_float2(1.f, 1.f);
            if (weight) {  // warp-uniform
                const float2 q = ffma2(y[1], y[1], ffma2(y[0], y[0], ffma2(x[1], x[1], fmul2(x[0], x[0]))));
                float ss = q.x + q.y;
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                inv.x = inv.y = rsqrtf(fmaf(ss, 1.0f / D, eps));
            }
            float2 u[2], v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (rot) {
                    u[i] = ffma2(y[i], t.ys[i], fmul2(x[i], t.xc[i]));
                    v[i] = ffma2(x[i], t.xs[i], fmul2(y[i], t.yc[i]));
                } else {  // xc and yc are the weights: cos 1, and no product that an infinity could spoil
                    u[i] = fmul2(x[i], t.xc[i]);
                    v[i] = fmul2(y[i], t.yc[i]);
                }
                u[i] = fmul2(u[i], inv);
                v[i] = fmul2(v[i], inv);
            }
            if (ok) {
                __nv_bfloat16 *o = dst + (p + j) * kRows * D;
                uint2 oa, ob;
                if (kInterleaved) {
                    oa = make_uint2(pack_bf16x2(u[0].x, v[0].x), pack_bf16x2(u[0].y, v[0].y));
                    ob = make_uint2(pack_bf16x2(u[1].x, v[1].x), pack_bf16x2(u[1].y, v[1].y));
                } else {
                    oa = make_uint2(pack_bf16x2(u[0].x, u[0].y), pack_bf16x2(u[1].x, u[1].y));
                    ob = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
                }
                *reinterpret_cast<uint2 *>(o + ea) = oa;
                *reinterpret_cast<uint2 *>(o + eb) = ob;
            }
        }
    }
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(32 * kRotWarps) qk_norm_rope_kernel(const RotaryArgs a) {
    constexpr int kLanes = D / 8;       // lanes of a row
    constexpr int kRows = 32 / kLanes;  // rows of a pass
    __shared__ float2 s_cs[kRotWarps][D / 2];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int l = lane % kLanes, row_in_pass = lane / kLanes;
    const int passes_q = a.q ? (a.Hq + kRows - 1) / kRows : 0;
    const int passes = passes_q + (a.k ? (a.Hkv + kRows - 1) / kRows : 0);
    const int64_t unit = (int64_t)blockIdx.x * kRotWarps + wid;
    const int64_t t = unit / a.splits;
    const int part = (int)(unit % a.splits);
    if (t >= a.T) return;  // warp-uniform; no block-wide barrier follows
    const int per = (passes + a.splits - 1) / a.splits;
    const int p_begin = part * per, p_end = min(passes, p_begin + per);
    const int R = a.rotary_dim;
    const int pos = R > 0 ? a.positions[t] : 0;
    if (pos < 0) return;  // padding: the token's rows are left as they were
    if (pos >= kRotaryMaxPos) {
        if (lane == 0 && part == 0) set_status(a.status, SINKATTN_STATUS_BAD_LENGTH);
        return;
    }
    // chunks of 4 elements: the lane's two, and whether they turn (in the half layout the
    // elements from R on are chunks 2l and 2l + 1 of the lanes from R / 8 on)
    const bool rot = l < R / 8;
    const int ea = 4 * (kInterleaved || !rot ? 2 * l : l);
    const int eb = 4 * (kInterleaved || !rot ? 2 * l + 1 : l + R / 8);
    for (int i = lane; i < R / 2; i += 32) s_cs[wid][i] = rope_cs((float)pos, a.hi[i], a.lo[i], a.mscale);
    __syncwarp();
    float2 cs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = rot ? s_cs[wid][4 * l + i] : make_float2(1.f, 0.f);
    run_rows<D, kInterleaved>(reinterpret_cast<const __nv_bfloat16 *>(a.q) + t * a.q_stride,
                              reinterpret_cast<__nv_bfloat16 *>(a.q_out) + t * a.Hq * D, a.Hq, p_begin,
                              min(p_end, passes_q), a.q_weight, a.eps, cs, rot, ea, eb, row_in_pass);
    run_rows<D, kInterleaved>(reinterpret_cast<const __nv_bfloat16 *>(a.k) + t * a.k_stride,
                              reinterpret_cast<__nv_bfloat16 *>(a.k_out) + t * a.Hkv * D, a.Hkv,
                              max(p_begin - passes_q, 0), p_end - passes_q, a.k_weight, a.eps, cs, rot, ea, eb,
                              row_in_pass);
}

template <int D>
cudaError_t launch_rotary_d(RotaryArgs a, cudaStream_t stream) {
    int sms = 0;
    const cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess) return e;
    constexpr int kRows = 32 / (D / 8);
    const int passes = (a.q ? (a.Hq + kRows - 1) / kRows : 0) + (a.k ? (a.Hkv + kRows - 1) / kRows : 0);
    // one warp per token while there are enough tokens to fill the GPU; with fewer, a token's
    // passes are split over several warps, a batch of loads each (128 tokens of 68 rows of 128:
    // 3.8 us, a single pass a warp 7.8: each warp computes its token's angles again)
    const int64_t want = (int64_t)sms * 32;
    int64_t splits = (want + a.T - 1) / a.T;
    const int64_t most = (passes + kRotBatch - 1) / kRotBatch;
    if (splits > most) splits = most;
    const int64_t per = (passes + splits - 1) / splits;
    a.splits = (int)((passes + per - 1) / per);
    const int64_t units = (int64_t)a.T * a.splits;
    const int64_t grid = (units + kRotWarps - 1) / kRotWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (a.interleaved)
        qk_norm_rope_kernel<D, true><<<(unsigned)grid, 32 * kRotWarps, 0, stream>>>(a);
    else
        qk_norm_rope_kernel<D, false><<<(unsigned)grid, 32 * kRotWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(int D, const RotaryArgs &a, cudaStream_t stream) {
    if (a.T <= 0 || (!a.q && !a.k)) return cudaSuccess;
    if (D == 64) return launch_rotary_d<64>(a, stream);
    if (D == 128) return launch_rotary_d<128>(a, stream);
    return cudaErrorInvalidValue;
}

}  // namespace sinkattn
