// Append into an INT8 paged cache with one scale for each page and KV head: new bf16 K/V rows
// are quantised into their pages, and a page that was already begun is brought to the scale its
// new rows need.
//
// For the new rows of one (page, KV head), amax their largest finite magnitude:
//     cand = amax / 127 rounded up to 8 significant bits
//     s'   = cand if the page starts with these rows, else max(s, cand)
//     code = rint(x / s') in [-127, 127];  codes of the page's earlier slots: rint(c * s / s')
// Scales of 8 significant bits, like the bf16 values themselves, make every quotient x / s' an
// exact tie or at least 2^-10 away from one: x * (1 / s'), snapped to multiples of 2^-11, then
// rounds exactly as the quotient does, without a division per element.
//
// Bound by HBM for long appends (4 D bytes read and 2 D written per token and head; 11708 tokens of 8
// heads of 64 take 8.5 us, 62 % of the copy rate) and by latency for a decode step's single tokens (64
// of them 3.4 us: entry, scale, rows, store one after the other).  A warp holds the new rows of one page and head, K
// and V (at most 2 x 16 x D bf16), in registers: their maxima, then their codes, in one pass
// over the data.  Which tokens begin a page's rows ("leaders") is found by the warp that owns
// the token, so no plan of the ragged batch is needed: a warp owns a group of consecutive
// tokens for one head, its lanes look the tokens up side by side, and it serves the leaders
// among them.
#include "internal.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

constexpr int kI8Warps = 4;
constexpr int kI8StageReqs = 1024;  // requests whose cu_seqlens / start_pos a block stages
// Scales below this (values below ~1e-28) are taken as zero: their reciprocals stay finite.
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ float scale_for(float amax) {
    const float y = __fdiv_rn(amax, 127.f);
    const float s = __uint_as_float((__float_as_uint(y) + 0xFFFFu) & 0xFFFF0000u);
    return s >= kScaleFloor ? s : 0.f;
}

// x * r rounded to a multiple of 2^-11, then to an integer (ties to even); the low byte of the
// result is its two's complement.  |x * r| <= 127.
__device__ __forceinline__ uint32_t code_of(float x, float r) {
    const float q = fmaf(x, r, 6144.f) - 6144.f;  // 1.5 * 2^12: unit in the last place 2^-11
    return __float_as_uint(q + 12582912.f);       // 1.5 * 2^23: unit in the last place 1
}

__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float r) {
    const uint32_t a = code_of(__uint_as_float(w0 << 16), r), b = code_of(__uint_as_float(w0 & 0xFFFF0000u), r);
    const uint32_t c = code_of(__uint_as_float(w1 << 16), r), d = code_of(__uint_as_float(w1 & 0xFFFF0000u), r);
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A bf16 (its 16 bits) as a float, NaN as 0 and infinities as the largest finite value.
__device__ __forceinline__ float finite_of(uint32_t x) {
    x &= 0xFFFFu;
    if ((x & 0x7FFFu) > 0x7F80u) x = 0;
    else if ((x & 0x7FFFu) == 0x7F80u) x = (x & 0x8000u) | 0x7F7Fu;
    return __uint_as_float(x << 16);
}

// Largest finite |x| of the warp's rows; `bad` if some element is not finite.
template <int N>
__device__ __forceinline__ float rows_amax(const uint4 (&x)[N], bool &bad) {
    uint32_t mx = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        mx = __vmaxu2(mx, x[e].x & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, x[e].y & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, x[e].z & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, x[e].w & 0x7FFF7FFFu);
    }
    uint32_t m = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
    bad = m >= 0x7F80u;
    if (bad) {  // rare: look again for the largest finite one
        m = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const uint32_t u[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v = (u[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
                if (v < 0x7F80u) m = max(m, v);
            }
        }
        m = __reduce_max_sync(0xffffffffu, m);
    }
    return __uint_as_float(m << 16);
}

// The rows of one tensor for one (page, head): scale, codes of the new rows, and the earlier
// slots' codes brought to a larger scale.  base: the (page, head)'s first code.
template <int D, int N>
__device__ __forceinline__ float put_rows(const uint4 (&x)[N], uint8_t *base, int slot0, int ntok, float s_old,
                                          int lane, uint32_t *status) {
    constexpr int kVec = D / 8;  // 16-byte vectors of a row
    bool bad;
    const float cand = scale_for(rows_amax<N>(x, bad));
    if (bad && lane == 0) set_status(status, SINKATTN_STATUS_VALUE_RANGE);
    const float before = slot0 > 0 && s_old >= kScaleFloor ? s_old : 0.f;
    const float s = fmaxf(before, cand);
    const float r = s > 0.f ? 1.0f / s : 0.f;
    if (slot0 > 0 && s > before) {
        // slots 0 .. slot0 - 1 to the new scale, 16 codes a lane and step
        for (int i = lane; i < slot0 * (D / 16); i += 32) {
            uint4 *p = reinterpret_cast<uint4 *>(base) + i;
            const uint4 w = *p;
            uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t o = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float c = (float)(int8_t)(u[e] >> (8 * b));
                    o |= ((uint32_t)__float2int_rn(__fdiv_rn(c * before, s)) & 0xFFu) << (8 * b);
                }
                u[e] = o;
            }
            *p = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int i = e * 32 + lane, row = i / kVec, c = i % kVec;
        if (row < ntok) {
            uint2 o = make_uint2(codes4(x[e].x, x[e].y, r), codes4(x[e].z, x[e].w, r));
            if (bad) {  // infinities at the end of the range, NaN as 0
                const uint32_t u[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
                uint32_t z[2] = {0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float q = fminf(fmaxf(finite_of(u[j >> 1] >> (16 * (j & 1))) * r, -127.f), 127.f);
                    z[j >> 2] |= (code_of(q, 1.f) & 0xFFu) << (8 * (j & 3));
                }
                o = make_uint2(z[0], z[1]);
            }
            *reinterpret_cast<uint2 *>(base + (slot0 + row) * D + c * 8) = o;
        }
    }
    return s;
}

template <int D>
__global__ void __launch_bounds__(32 * kI8Warps) append_int8_kernel(const AppendInt8Args a) {
    constexpr int kVec = D / 8;
    constexpr int N = kPageSize * kVec / 32;  // vectors a lane holds of K, and of V
    __shared__ int s_cu[kI8StageReqs + 1];
    __shared__ int s_start[kI8StageReqs];
    const bool staged = a.n <= kI8StageReqs;
    if (staged) {
        for (int i = threadIdx.x; i <= a.n; i += blockDim.x) {
            s_cu[i] = a.cu_seqlens[i];
            if (i < a.n) s_start[i] = a.start_pos[i];
        }
    }
    __syncthreads();
    const int *cu = staged ? s_cu : a.cu_seqlens;
    const int *sp = staged ? s_start : a.start_pos;
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kI8Warps + (threadIdx.x >> 5);
    const int g = (int)(unit % a.Hkv);
    const int64_t first = unit / a.Hkv * a.group;  // the warp's tokens: first .. first + group - 1
    if (first >= a.T) return;

    // one token per lane: its request, position, page, and whether it begins a page's rows
    const int64_t t = first + lane;
    bool leader = false;
    int slot0 = 0, ntok = 0, pg = -1;
    if (lane < a.group && t < a.T) {
        int lo = 0, hi = a.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int c0 = cu[lo], c1 = min(cu[lo + 1], a.T);
        uint32_t bad = 0;
        if (t < c0 || t >= c1) {
            bad = SINKATTN_STATUS_BAD_CU_SEQLENS;
        } else {
            const int64_t pos = (int64_t)sp[lo] + (t - c0);
            if (pos < 0 || pos / kPageSize >= a.max_pages) {
                bad = SINKATTN_STATUS_BAD_LENGTH;
            } else if (t == c0 || pos % kPageSize == 0) {
                slot0 = (int)(pos % kPageSize);
                ntok = min(kPageSize - slot0, (int)(c1 - t));
                pg = a.block_table[(int64_t)lo * a.max_pages + pos / kPageSize];
                leader = true;
            }
        }
        if (bad && g == 0) set_status(a.status, bad);
    }
    uint32_t leaders = __ballot_sync(0xffffffffu, leader);
    for (; leaders; leaders &= leaders - 1) {
        const int src = __ffs(leaders) - 1;
        const int s0 = __shfl_sync(0xffffffffu, slot0, src), nt = __shfl_sync(0xffffffffu, ntok, src);
        const __nv_bfloat16 *kr = reinterpret_cast<const __nv_bfloat16 *>(a.k) + (first + src) * a.k_stride + (int64_t)g * D;
        const __nv_bfloat16 *vr = reinterpret_cast<const __nv_bfloat16 *>(a.v) + (first + src) * a.v_stride + (int64_t)g * D;
        uint4 kx[N], vx[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int i = e * 32 + lane, row = i / kVec, c = i % kVec;
            kx[e] = vx[e] = make_uint4(0, 0, 0, 0);
            if (row < nt) {
                kx[e] = *reinterpret_cast<const uint4 *>(kr + row * a.k_stride + c * 8);
                vx[e] = *reinterpret_cast<const uint4 *>(vr + row * a.v_stride + c * 8);
            }
        }
        // the rows are on their way before the page's entry is needed
        const int64_t page = __shfl_sync(0xffffffffu, pg, src);
        if (page < 0 || page >= a.num_pages) {  // warp-uniform
            if (lane == 0 && g == 0) set_status(a.status, SINKATTN_STATUS_BAD_PAGE);
            continue;
        }
        float2 *sc = reinterpret_cast<float2 *>(a.kv_scales) + page * a.Hkv + g;
        const float2 old = s0 > 0 ? *sc : make_float2(0.f, 0.f);
        const int64_t at = (page * a.Hkv + g) * kPageSize * D;
        const float ks = put_rows<D, N>(kx, static_cast<uint8_t *>(a.k_pages) + at, s0, nt, old.x, lane, a.status);
        const float vs = put_rows<D, N>(vx, static_cast<uint8_t *>(a.v_pages) + at, s0, nt, old.y, lane, a.status);
        __syncwarp();  // every lane has read the old scales
        if (lane == 0) *sc = make_float2(ks, vs);
    }
}

}  // namespace

cudaError_t launch_append_int8(int D, AppendInt8Args a, cudaStream_t stream) {
    if (a.T <= 0 || a.Hkv <= 0) return cudaSuccess;
    int sms = 0;
    const cudaError_t e = current_sms(&sms);
    if (e != cudaSuccess) return e;
    // a page's worth of tokens a warp once that still fills the GPU, else one token a warp: 11708
    // tokens of 8 heads of 64 take 8.5 us so and 33 us with a token a warp, whose lanes find out for
    // one token what they could for sixteen
    a.group = (int64_t)a.T * a.Hkv > (int64_t)sms * 64 ? kPageSize : 1;
    const int64_t units = ((int64_t)a.T + a.group - 1) / a.group * a.Hkv;
    const int64_t grid = (units + kI8Warps - 1) / kI8Warps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (D == 64)
        append_int8_kernel<64><<<(unsigned)grid, 32 * kI8Warps, 0, stream>>>(a);
    else if (D == 128)
        append_int8_kernel<128><<<(unsigned)grid, 32 * kI8Warps, 0, stream>>>(a);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace sinkattn
