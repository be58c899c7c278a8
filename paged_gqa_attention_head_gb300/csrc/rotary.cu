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
// Bound by HBM: 2 D bytes in and 2 D out per row, ~130 instructions per 2 KB moved.  A row is
// held by D/16 lanes, each with two 16-byte chunks whose pairs it can turn alone: chunks c and
// c + R/16 in the half layout, two neighbours in the interleaved one.  So a row needs no
// exchange beyond the norm's 2 or 3 shuffles, a warp moves 512 elements a pass, and every
// 32-byte sector it touches is used whole.  The angles depend on the token only: a warp
// works for one token, takes its R/2 (cos, sin) once into shared memory (one or two sincos per
// lane) and uses them for all of its rows.
#include "internal.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace sinkattn {
namespace {

constexpr int kRotWarps = 4;

struct RowBits {
    uint4 a, b;
};

__device__ __forceinline__ void unpack8(const uint4 &w, float *x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}

template <int D>
__global__ void __launch_bounds__(32 * kRotWarps) qk_norm_rope_kernel(const RotaryArgs a) {
    constexpr int kLanes = D / 16;      // lanes of a row
    constexpr int kRows = 32 / kLanes;  // rows of a pass
    constexpr int kBatch = 4;           // passes whose loads are issued together
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
    // chunks of 8 elements: the lane's two, and whether they turn (in the half layout the
    // elements from R on are chunks 2l and 2l + 1 of the lanes from R / 16 on)
    const int rot_lanes = R / 16;
    const bool rot = l < rot_lanes;
    const int ca = a.interleaved || !rot ? 2 * l : l;
    const int cb = a.interleaved || !rot ? 2 * l + 1 : l + rot_lanes;

    RowBits x[kBatch];
    auto row_of = [&](int p, int &h, bool &is_k) {
        is_k = p >= passes_q;
        h = (is_k ? p - passes_q : p) * kRows + row_in_pass;
        return h < (is_k ? a.Hkv : a.Hq);
    };
    auto load = [&](int p0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            int h;
            bool is_k;
            if (p0 + j < p_end && row_of(p0 + j, h, is_k)) {
                const __nv_bfloat16 *src = is_k ? reinterpret_cast<const __nv_bfloat16 *>(a.k) + t * a.k_stride
                                                : reinterpret_cast<const __nv_bfloat16 *>(a.q) + t * a.q_stride;
                src += (int64_t)h * D;
                x[j].a = *reinterpret_cast<const uint4 *>(src + ca * 8);
                x[j].b = *reinterpret_cast<const uint4 *>(src + cb * 8);
            } else {
                x[j].a = x[j].b = make_uint4(0, 0, 0, 0);
            }
        }
    };
    load(p_begin);
    if (pos < 0) return;  // padding: the token's rows are left as they were
    if (pos >= kRotaryMaxPos) {
        if (lane == 0 && part == 0) set_status(a.status, SINKATTN_STATUS_BAD_LENGTH);
        return;
    }
    for (int i = lane; i < R / 2; i += 32) s_cs[wid][i] = rope_cs((float)pos, a.hi[i], a.lo[i], a.mscale);
    __syncwarp();
    float2 cs[8];
    if (rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = s_cs[wid][8 * l + i];
    }
    float w[16];
    int have = -1;  // whose weights w holds: 0 q, 1 k
    for (int p0 = p_begin; p0 < p_end; p0 += kBatch) {
        if (p0 > p_begin) load(p0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            int h;
            bool is_k;
            if (p0 + j >= p_end) break;
            const bool ok = row_of(p0 + j, h, is_k);
            const float *wt = is_k ? a.k_weight : a.q_weight;
            float v[16];
            unpack8(x[j].a, v);
            unpack8(x[j].b, v + 8);
            if (wt) {  // warp-uniform
                if (have != (int)is_k) {
                    have = is_k;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = __ldg(reinterpret_cast<const float4 *>(wt + (i < 2 ? ca : cb) * 8) + (i & 1));
                        w[4 * i] = f.x;
                        w[4 * i + 1] = f.y;
                        w[4 * i + 2] = f.z;
                        w[4 * i + 3] = f.w;
                    }
                }
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = v[i] * inv * w[i];
            }
            if (rot) {
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float e = v[2 * i], f = v[2 * i + 1];
                        v[2 * i] = fmaf(e, cs[i].x, -(f * cs[i].y));
                        v[2 * i + 1] = fmaf(f, cs[i].x, e * cs[i].y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float e = v[i], f = v[i + 8];
                        v[i] = fmaf(e, cs[i].x, -(f * cs[i].y));
                        v[i + 8] = fmaf(f, cs[i].x, e * cs[i].y);
                    }
                }
            }
            if (ok) {
                __nv_bfloat16 *dst = is_k ? reinterpret_cast<__nv_bfloat16 *>(a.k_out) + t * a.Hkv * D
                                          : reinterpret_cast<__nv_bfloat16 *>(a.q_out) + t * a.Hq * D;
                dst += (int64_t)h * D;
                *reinterpret_cast<uint4 *>(dst + ca * 8) = pack8(v);
                *reinterpret_cast<uint4 *>(dst + cb * 8) = pack8(v + 8);
            }
        }
    }
}

template <int D>
cudaError_t launch_rotary_d(RotaryArgs a, cudaStream_t stream) {
    int device = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device)) != cudaSuccess) return e;
    constexpr int kRows = 32 / (D / 16);
    const int passes = (a.q ? (a.Hq + kRows - 1) / kRows : 0) + (a.k ? (a.Hkv + kRows - 1) / kRows : 0);
    // one warp per token while there are enough tokens to fill the GPU; with fewer, a token's
    // passes are split over several warps
    const int64_t want = (int64_t)sms * 32;
    int64_t splits = (want + a.T - 1) / a.T;
    if (splits > passes) splits = passes;
    const int64_t per = (passes + splits - 1) / splits;
    a.splits = (int)((passes + per - 1) / per);
    const int64_t units = (int64_t)a.T * a.splits;
    const int64_t grid = (units + kRotWarps - 1) / kRotWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    qk_norm_rope_kernel<D><<<(unsigned)grid, 32 * kRotWarps, 0, stream>>>(a);
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
