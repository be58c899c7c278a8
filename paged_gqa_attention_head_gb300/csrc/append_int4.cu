// The 4-bit paged cache: new bf16 K/V rows quantised into their slots, and pages back as the bf16
// values that they stand for.
//
// A group is 32 channels of one token, so an appended row touches no other token's codes, and a
// row's slot is all that the kernel has to know of the batch.  For a group with low = min(0, min x)
// and high = max(0, max x):
//     s    = the smallest number of four significant bits with 15 s >= high - low
//     z    = rint(-low / s),   code = min(15, rint(x / s + z)),   value = s (code - z)
// A scale and a code difference of four bits each make every value a bf16 number.  Quotients of
// bf16 values by such a scale are exact ties or at least 2^-11 away from one: x * (1 / s) + z,
// snapped to multiples of 2^-11, then rounds exactly as the quotient does.
//
// Record of a (page, KV head, K or V), 9 D bytes: codes [D / 32 groups][16 tokens][16 bytes], then
// [D / 32][16] 16-bit words, the bf16 scale with z in its low four bits.  The codes lie so that
// 8x8 loads of a group's rows meet no bank conflict, and eight channels of a token in one 32-bit
// word, channel c at bit 4 (c / 2) + 16 (c % 2): masking a word with 0x000f000f leaves a pair of
// neighbouring channels, or, after a transposing load, one channel of two neighbouring tokens.
//
// Bound by HBM and instruction issue alike for long appends and for unpacking, by latency for a decode step.  A
// warp holds eight tokens of one head, four lanes to a group, all groups of K and V at once: reads of 64 bytes
// and, where the tokens' slots follow each other, writes of 128.  Measured: 16381 tokens of 4 heads of 128
// appended in 9.5 us (4.5 TB/s, issue slots 0.63; 14.1 us with exact divisions and single elements in the
// range), their 1033 pages unpacked in 7.7 us (5.6 TB/s); 64 single tokens of 8 heads of 64 in 2.3 us.
#include "internal.h"
#include "ptx.cuh"

namespace sinkattn {
namespace {

constexpr int kI4Warps = 4;
constexpr float kScaleFloor4 = 7.888609052210118e-31f;  // 2^-100: smaller scales are taken as zero

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// min and max of bf16 pairs, NaN if either is.
__device__ __forceinline__ uint32_t min_bf2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Scale of a group of range high + below (low = -below): the smallest s of four significant bits with
// 7.5 s >= half the range (halved, so that it cannot overflow, and rounded upwards: it passes 7.5 s, eight
// bits, if and only if the exact one does).  Half the range times 1/7.5, both rounded upwards, is no
// less than the quotient and at most a rounding more, so its next number of four bits is s or the one above.
__device__ __forceinline__ float scale4(float below, float high) {
    const float half = __fadd_ru(0.5f * high, 0.5f * below);
    const uint32_t up = (__float_as_uint(__fmul_ru(half, 0.13333334f)) + 0xFFFFFu) & 0xFFF00000u;
    const float under = __uint_as_float(up - 0x100000u);
    const float s = 7.5f * under >= half ? under : __uint_as_float(up);
    return s >= kScaleFloor4 ? s : 0.f;
}
static_assert(0.13333334f >= 1.0 / 7.5, "1/7.5 rounded upwards");

// x r + z, snapped to multiples of 2^-11 by the exponent of z6144 = 6144 + z (1.5 * 2^12), then rounded:
// the integer in the low bits.  (An approximate reciprocal will do: the snap takes off up to 2^-12.)
__device__ __forceinline__ uint32_t code4(float x, float r, float z6144) {
    return __float_as_uint(fmaf(x, r, z6144) + (12582912.f - 6144.f));
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// High and -low of the finite elements among a lane's eight, as a bf16 pair.
__device__ __noinline__ uint32_t finite_range(uint4 x) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    float low = 0.f, high = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t v = (u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
        if ((v & 0x7FFFu) >= 0x7F80u) continue;
        low = fminf(low, __uint_as_float(v << 16));
        high = fmaxf(high, __uint_as_float(v << 16));
    }
    return pack_bf16x2(high, -low);
}
// The codes w with those of infinities and NaN put right: 15 and 0, and z.
__device__ __noinline__ uint32_t mend_codes(uint4 x, uint32_t w, uint32_t z) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t v = (u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
        const int bit = 4 * (i >> 1) + 16 * (i & 1);
        if ((v & 0x7FFFu) < 0x7F80u) continue;
        const uint32_t code = (v & 0x7FFFu) > 0x7F80u ? z : v & 0x8000u ? 0u : 15u;
        w = (w & ~(15u << bit)) | code << bit;
    }
    return w;
}

// Eight channels of one lane and their group's word; the four lanes of a group call it together.
__device__ __forceinline__ uint32_t quantise8(const uint4 &x, uint32_t &word, bool &bad) {
    const uint32_t lo2 = min_bf2(min_bf2(x.x, x.y), min_bf2(x.z, x.w));
    const uint32_t hi2 = max_bf2(max_bf2(x.x, x.y), max_bf2(x.z, x.w));
    // (high, -low) as a pair, 0 counted in
    uint32_t span = max_bf2(max_bf2(__byte_perm(hi2, lo2 ^ 0x80008000u, 0x5410), __byte_perm(hi2, lo2 ^ 0x80008000u, 0x7632)), 0u);
    span = max_bf2(span, __shfl_xor_sync(0xffffffffu, span, 1));
    span = max_bf2(span, __shfl_xor_sync(0xffffffffu, span, 2));
    bad = (span & 0x7F80u) == 0x7F80u || (span & 0x7F800000u) == 0x7F800000u;  // all four lanes alike
    if (__any_sync(0xffffffffu, bad)) {
        uint32_t fin = finite_range(x);
        fin = max_bf2(fin, __shfl_xor_sync(0xffffffffu, fin, 1));
        fin = max_bf2(fin, __shfl_xor_sync(0xffffffffu, fin, 2));
        if (bad) span = fin;
    }
    const float below = bf_hi(span), s = scale4(below, bf_lo(span));
    const float r = s > 0.f ? rcp_approx(s) : 0.f;
    const uint32_t z = code4(below, r, 6144.f) & 15u;
    word = (__float_as_uint(s) >> 16) | z;
    const float zf = (float)z + 6144.f;
    uint32_t w = 0;
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = code4(bf_lo(u[i]), r, zf), b = code4(bf_hi(u[i]), r, zf);
        w |= __vminu2(__byte_perm(a, b, 0x5410), 0x000F000Fu) << (4 * i);
    }
    if (bad) w = s > 0.f ? mend_codes(x, w, z) : 0u;
    return w;
}

template <int D>
__global__ void __launch_bounds__(32 * kI4Warps) append_int4_kernel(const AppendInt4Args a) {
    constexpr int NG = D / 32;
    const int lane = threadIdx.x & 31, t4 = lane & 3;
    const int64_t unit = (int64_t)blockIdx.x * kI4Warps + (threadIdx.x >> 5);
    const int g = (int)(unit % a.Hkv);
    const int64_t t = unit / a.Hkv * 8 + (lane >> 2);
    if (unit / a.Hkv * 8 >= a.T) return;
    const bool in = t < a.T;
    uint4 x[2][NG];
    const __nv_bfloat16 *kr = reinterpret_cast<const __nv_bfloat16 *>(a.k) + t * a.k_stride + (int64_t)g * D + 8 * t4;
    const __nv_bfloat16 *vr = reinterpret_cast<const __nv_bfloat16 *>(a.v) + t * a.v_stride + (int64_t)g * D + 8 * t4;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        x[0][i] = x[1][i] = make_uint4(0, 0, 0, 0);
        if (in) {
            x[0][i] = __ldg(reinterpret_cast<const uint4 *>(kr + 32 * i));
            x[1][i] = __ldg(reinterpret_cast<const uint4 *>(vr + 32 * i));
        }
    }
    int64_t slot = in ? a.slots[t] : -1;
    const int64_t page = slot / kPageSize;
    if (slot >= 0 && page >= a.num_pages) {
        if (g == 0 && t4 == 0) set_status(a.status, SINKATTN_STATUS_BAD_PAGE);
        slot = -1;
    }
    const int tok = (int)(slot % kPageSize);
    uint8_t *rec = static_cast<uint8_t *>(a.kv_pages) + (page * a.Hkv + g) * (18 * D);
    bool any_bad = false;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            uint32_t word;
            bool bad;
            const uint32_t codes = quantise8(x[kv][i], word, bad);
            any_bad |= bad;
            if (slot >= 0) {
                uint8_t *r = rec + kv * 9 * D;
                *reinterpret_cast<uint32_t *>(r + (i * kPageSize + tok) * 16 + 4 * t4) = codes;
                if (t4 == 0) *reinterpret_cast<uint16_t *>(r + 8 * D + (i * kPageSize + tok) * 2) = (uint16_t)word;
            }
        }
    if (any_bad && slot >= 0) set_status(a.status, SINKATTN_STATUS_VALUE_RANGE);
}

__device__ __forceinline__ uint32_t sub_bf2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A thread takes a run of eight channels of a token, D / 8 neighbouring threads a row: 16-byte stores
// side by side, and 64 bytes of codes of each group to a warp.
template <int D>
__global__ void __launch_bounds__(256) unpack_int4_kernel(const UnpackInt4Args a) {
    constexpr int kRuns = D / 8, kPer = 2 * kPageSize * kRuns;  // runs of a row; of a (page, head)
    const uint32_t pairs = (uint32_t)a.n * a.Hkv;  // (page, head) pairs, below 2^31
    constexpr int N = 4;
    uint32_t w[N], p[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const uint32_t i = e * 256 + threadIdx.x, ph = blockIdx.x * (256 * N / kPer) + i / kPer;
        w[e] = p[e] = 0;
        if (ph >= pairs) continue;
        const int at = (int)(i % kPer), kv = at / (kPageSize * kRuns), tok = at / kRuns % kPageSize, c = at % kRuns;
        const uint32_t head = ph % (uint32_t)a.Hkv;
        int64_t page = ph / (uint32_t)a.Hkv;
        if (a.pages) page = a.pages[page];
        if (page < 0 || page >= a.num_pages) {
            if (at == 0 && head == 0) set_status(a.status, SINKATTN_STATUS_BAD_PAGE);
            continue;  // its values are zeros
        }
        const uint8_t *r = static_cast<const uint8_t *>(a.kv_pages) + ((page * a.Hkv + head) * 2 + kv) * (9 * D);
        const int row = c / 4 * kPageSize + tok;
        w[e] = __ldg(reinterpret_cast<const uint32_t *>(r + row * 16 + 4 * (c % 4)));
        p[e] = __ldg(reinterpret_cast<const uint16_t *>(r + 8 * D + 2 * row));
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const uint32_t i = e * 256 + threadIdx.x, ph = blockIdx.x * (256 * N / kPer) + i / kPer;
        if (ph >= pairs) continue;
        const int at = (int)(i % kPer), kv = at / (kPageSize * kRuns), rest = at % (kPageSize * kRuns);
        // 128 + code and 128 + z are bf16 numbers, and so is all that follows
        const uint32_t s = (p[e] & 0xFFF0u) * 0x10001u, z = (p[e] & 15u) * 0x10001u + 0x43004300u;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = mul_bf2(sub_bf2(((w[e] >> (4 * j)) & 0x000F000Fu) | 0x43004300u, z), s);
        __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(kv ? a.v_out : a.k_out);
        *reinterpret_cast<uint4 *>(out + ((int64_t)ph * (kPageSize * kRuns) + rest) * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

cudaError_t launch_append_int4(int D, const AppendInt4Args &a, cudaStream_t stream) {
    if (a.T <= 0 || a.Hkv <= 0) return cudaSuccess;
    const int64_t units = ((int64_t)a.T + 7) / 8 * a.Hkv, grid = (units + kI4Warps - 1) / kI4Warps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (D == 64)
        append_int4_kernel<64><<<(unsigned)grid, 32 * kI4Warps, 0, stream>>>(a);
    else if (D == 128)
        append_int4_kernel<128><<<(unsigned)grid, 32 * kI4Warps, 0, stream>>>(a);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

cudaError_t launch_unpack_int4(int D, const UnpackInt4Args &a, cudaStream_t stream) {
    const int64_t pairs = (int64_t)a.n * a.Hkv, per = 1024 / (4 * D), grid = (pairs + per - 1) / per;
    if (grid <= 0) return cudaSuccess;
    if (pairs > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (D == 64)
        unpack_int4_kernel<64><<<(unsigned)grid, 256, 0, stream>>>(a);
    else if (D == 128)
        unpack_int4_kernel<128><<<(unsigned)grid, 256, 0, stream>>>(a);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace sinkattn
