// Split-KV paged decode with per-head sinks over an INT8 cache with one scale for each page and
// KV head (element value = s(page, g) * code; one fp32 pair of scales, K and V).
//
// The plan, the copies and the products are those of the FP8 decode: every warp takes an equal
// run of two-page units, S^T = K Q^T and O^T = V^T P^T on m16n8k16 f16 MMAs with the 16 tokens of
// a page, then head_dim, on the M axis and the query heads on N; the contraction index permuted so
// that a lane's K fragment is one run of D/4 bytes; V comes by transposing 8x8 loads of its byte
// pairs, which lay the pair of one lane's two tokens beside each other.
// What the scales and the codes change:
//   * a code is taken as the f16 subnormal (code + 128) 2^-24, whose bits are the code's with the
//     sign flipped: one AND-XOR for two codes (a shift more for the other two of a word).  The
//     128 comes off in the MMAs' accumulators: the K products start from -128 2^-24 sum(q), and
//     what the P of a unit add too much is one MMA of a constant -128 2^-24 against them, added to
//     O^T.  (As values - the offset form under the exponent of 1024, less 1152 - a page cost 27
//     instructions more at head_dim 64.)  The detour through 128 makes the fp32 sums' rounding that of
//     sums of codes of 128 to 255: it costs a channel of full range a bit, one whose codes are a few
//     units beside an outlier channel's up to seven of its 24, where P keeps 11;
//   * K: a page's scale multiplies its 16 scores, together with the softmax scale;
//   * V: P of a page is taken times s / 2^E, with 2^E the power of two above the largest V scale
//     the warp has met in this (sequence, head): one rounding to f16, and O^T is summed in the
//     MMA's fp32 accumulators over all pages.  When a larger scale comes, O^T and E move by
//     an exact power of two.  (Taking each page's product apart and adding it with an FMA per
//     element rounds no scale at all, and cost 64 FMAs a page at head_dim 128 and 16 heads,
//     a tenth of the instructions.  Rounding P times the scale is as exact as rounding P for
//     products within 2^20 of the largest, and beyond that is off by 2^-31 of it: the largest is
//     2^6 or more, f16 subnormals end at 2^-24.)
//   * q times a power of two per (sequence, KV head) that puts its largest entry at 2^14 is exact
//     in f16 whatever its size; the scores take the power back;
//   * no code is NaN or infinite: slots past a sequence's end need no clearing, P is 0 there.
// A warp's copy side runs ahead of its arithmetic and leaves what that needs to know of a unit
// beside its pages.
// The running maximum moves only when a score passes it by more than 8 (log2): P is taken as
// 2^(s - m + 7), at most 2^15, so a stale maximum costs no precision and the votes, the column
// maxima and the rescale of O^T drop out of almost every unit.
// Measured: 64 sequences up to 131072 tokens, 64/8 heads of 64 (1.26 GB) 200 us, 6.3 TB/s, bound by
// HBM; 64 sequences up to 16384, 64/4 heads of 128 (0.56 GB) 109 us, 5.1 TB/s, bound by the latencies
// of the two warps a scheduler that the accumulators of 16 heads leave room for.
#include <math.h>

#include <mutex>
#include <vector>

#include "decode_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace sinkattn {

namespace {

template <int D, int NH>
struct Int8Cfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = kWarps * 32;
    // Pages per work unit: 8 KB of K and V (at head_dim 64 half of that for 16 heads, by registers).
    // What a unit costs beside its pages' arithmetic is ~300 instructions: with two pages at head_dim
    // 64 the batch of 1.26 GB ran 9 % longer.
    static constexpr int kPPU = D == 64 && NH == 1 ? 4 : 2;
    static constexpr int kStages = D == 64 && NH == 2 ? 4 : 2;
    static constexpr int kPageBytes = kPageSize * D;           // one (page, head) of K or of V codes
    static constexpr int kStageBytes = 2 * kPPU * kPageBytes;  // the unit's K pages, then V pages
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kKSteps = D / 16;  // S^T k-steps over head_dim
    static constexpr int kMTiles = D / 16;  // O^T m-tiles over head_dim
    static constexpr int kKWords = D / 16;  // 32-bit words of K a lane reads per token row
};

constexpr float kPShift = 7.f;   // P = 2^(s - m + kPShift)
constexpr float kMaxSlack = 8.f; // the running maximum moves when a score passes it by more
// A state leaves a warp with its sums over 2^(kPShift + kMaxSlack), the largest P, so that up to 2^17
// values of 2^107 (scales of 2^100) stay finite in it and in the merge.
constexpr float kStateDown = 1.f / 32768.f;

template <int D, int NH>
int int8_smem_bytes(int B) {
    using C = Int8Cfg<D, NH>;
    // per (warp, stage): its barrier, a UnitMeta, and a PageMeta for each page of its unit
    return 1024 /* alignment slack */ + C::kWarps * C::kWarpBytes + C::kWarps * C::kStages * (8 + 16 + 16 * C::kPPU) +
           (3 * B + 1) * 4;
}

// Byte offset of byte c of token t inside a page buffer.  A page's 16 x D contiguous bytes are
// copied as rows of 128 bytes (at head_dim 64 a row is two tokens: half the rows and requests) under
// the 128-byte swizzle, which keeps every shared load below free of bank conflicts.
template <int D>
__device__ __forceinline__ uint32_t page_off(int t, int c) {
    const int at = t * D + c;
    return sw128(at >> 7, (at >> 4) & 7) + (at & 15);
}

// What the arithmetic needs of a unit: whose it is, and of one of its pages.
struct __align__(16) UnitMeta {
    int b, g;   // sequence, KV head
    int flags;  // kStart | kEnd | kWhole
};
constexpr int kStart = 1, kEnd = 2, kWhole = 4;  // first / last unit of a segment; the segment is all of (b, g)
struct __align__(16) PageMeta {
    float ks, vs;  // K scale * 2^24, V scale (0 for a page that is not there)
    int nv, lo;    // its keys lo .. nv - 1 are visible
};

// Codes 0 and 2 (even) or 1 and 3 (odd) of a word as f16 pairs of (code + 128) 2^-24.
__device__ __forceinline__ uint32_t sub_even(uint32_t w) {
    uint32_t r;  // (w & mask) ^ sign in one instruction
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(0x00FF00FFu), "r"(0x00800080u));
    return r;
}
__device__ __forceinline__ uint32_t sub_odd(uint32_t w) { return sub_even(w >> 8); }
__device__ __forceinline__ uint32_t bf16x2_to_f16x2_times(uint32_t v, float mul) {
    return pack_f16x2(__uint_as_float(v << 16) * mul, __uint_as_float(v & 0xFFFF0000u) * mul);
}

constexpr uint32_t kMinus128 = 0x80808080u;  // an f16 pair of -128 * 2^-24
constexpr float kUp24 = 16777216.f;          // 2^24

// NH: 8-head tiles of the query group (1 for G <= 8, 2 for G = 16).
template <int D, int NH, bool kWindow>
__global__ void __launch_bounds__(Int8Cfg<D, NH>::kThreads, NH == 2 && D == 128 ? 2 : 3)
    decode_int8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const DecodeArgs a) {
    using C = Int8Cfg<D, NH>;
    constexpr int S = C::kStages, U = C::kPPU;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kWarps * C::kWarpBytes);
    UnitMeta *s_unit = reinterpret_cast<UnitMeta *>(bars + C::kWarps * S);     // [warp][stage]
    PageMeta *s_meta = reinterpret_cast<PageMeta *>(s_unit + C::kWarps * S);  // [warp][stage][page]
    int *s_prefix = reinterpret_cast<int *>(s_meta + C::kWarps * S * U);
    int *s_len = s_prefix + a.B + 1;
    int *s_first = s_len + a.B;

    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    if (lane < S) mbar_init(&bars[wid * S + lane], 1);
    fence_mbar_init();
    scan_pages<U>(a, s_prefix, s_len, s_first);  // contains __syncthreads

    const int64_t T = (int64_t)a.Hkv * s_prefix[a.B];
    int64_t per = (T + a.total_warps - 1) / a.total_warps;
    // at least 2 units a warp (16 heads: 4, whose partial states are four times the bytes of a unit's
    // share): one sequence of 4097 tokens took 10.5 us with 2, 12.6 with 4 and 11.3 with 1 at head_dim
    // 64, and 16.3 with 2, 15.8 with 4 at head_dim 128 and 16 heads
    constexpr int kMinUnits = NH == 1 ? 2 : 4;
    if (per < kMinUnits) per = kMinUnits;
    if (blockIdx.x == 0) {
        for (int b = tid; b <= a.B; b += blockDim.x) a.ws_prefix[b] = s_prefix[b];
        if (tid == 0) {
            a.ws_plan[0] = T;
            a.ws_plan[1] = per;
        }
    }
    const int wglob = blockIdx.x * C::kWarps + wid;
    const int64_t u_begin = (int64_t)wglob * per;
    if (u_begin >= T) return;  // warp-uniform; no block-wide barrier follows
    const int n_units = (int)min(per, T - u_begin);

    uint8_t *wbuf = smem + wid * C::kWarpBytes;
    uint64_t *wbar = bars + wid * S;
    UnitMeta *wunit = s_unit + wid * S;
    PageMeta *wmeta = s_meta + wid * S * U;

    // The copy side's position, the first unit of its segment, and the units copied so far.
    Cursor pc;
    {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            int mid = (lo + hi + 1) >> 1;
            if ((int64_t)a.Hkv * s_prefix[mid] <= u_begin)
                lo = mid;
            else
                hi = mid - 1;
        }
        pc.b = lo;
        pc.pb = s_prefix[lo + 1] - s_prefix[lo];
        const int local = (int)(u_begin - (int64_t)a.Hkv * s_prefix[lo]);
        pc.g = local / pc.pb;
        pc.p = local % pc.pb;
    }
    int p_seg0 = pc.p, produced = 0;

    // Block-table window: lane l holds the entry of visible page win_p0 + l of sequence
    // win_b (-1 past its last page) and that page's scales for KV head win_g; the entries of
    // the next 32 pages are loaded with it, and their scales halfway through it.
    int win_b = -1, win_p0 = 0, win_g = -1, win_val = -1, nxt_val = -1;
    float2 win_sc = make_float2(0.f, 0.f), nxt_sc = win_sc;
    bool nxt_ready = false;
    auto entry = [&](int b, int first, int npv, int q) {
        return q < npv ? a.block_table[(int64_t)b * a.max_pages + first + q] : -1;
    };
    auto scales = [&](int pg, int g) {
        return pg >= 0 && pg < a.num_pages
                   ? __ldg(reinterpret_cast<const float2 *>(a.kv_scales) + (int64_t)pg * a.Hkv + g)
                   : make_float2(0.f, 0.f);
    };
    const uint64_t policy = l2_policy_evict_first();
    // The next unit, if there is one, into a stage: lanes 0 .. U - 1 take a page each.
    auto produce = [&](int stage) {
        if (produced == n_units) return;
        const Cursor c = pc;
        ++produced;
        int flags = 0;
        if (c.p == p_seg0) flags |= kStart;
        if (c.p == c.pb - 1 || produced == n_units) flags |= kEnd;
        if (c.p == c.pb - 1 && p_seg0 == 0) flags |= kWhole;
        if (++pc.p == pc.pb) {
            pc.p = p_seg0 = 0;
            if (++pc.g == a.Hkv) {
                pc.g = 0;
                do {
                    ++pc.b;
                    pc.pb = pc.b < a.B ? s_prefix[pc.b + 1] - s_prefix[pc.b] : 1;
                } while (pc.b < a.B && pc.pb == 0);
            }
        }
        const int first = kWindow ? s_first[c.b] : 0;
        const int L = s_len[c.b];
        const int npv = (L + kPageSize - 1) / kPageSize - first;  // pages the query sees
        const int pp0 = c.p * U, p0 = pp0 & ~31;
        if (c.b != win_b || p0 != win_p0 || c.g != win_g) {  // warp-uniform
            if (nxt_ready && c.b == win_b && c.g == win_g && p0 == win_p0 + 32) {
                win_val = nxt_val;
                win_sc = nxt_sc;
            } else {
                if (c.b != win_b || p0 != win_p0) win_val = entry(c.b, first, npv, p0 + lane);
                win_sc = scales(win_val, c.g);
            }
            nxt_val = entry(c.b, first, npv, p0 + 32 + lane);
            nxt_ready = false;
            win_b = c.b;
            win_p0 = p0;
            win_g = c.g;
        } else if (!nxt_ready && pp0 - p0 >= 16) {
            nxt_sc = scales(nxt_val, c.g);
            nxt_ready = true;
        }
        const int src = (pp0 + (lane & (U - 1))) & 31;
        const int pg = __shfl_sync(0xffffffffu, win_val, src);
        const float ks = __shfl_sync(0xffffffffu, win_sc.x, src), vs = __shfl_sync(0xffffffffu, win_sc.y, src);
        const bool in = lane < U && pp0 + lane < npv, ok = in && pg >= 0 && pg < a.num_pages;
        if (in && !ok) set_status(a.status, SINKATTN_STATUS_BAD_PAGE);
        if (lane < U) {
            const int key0 = kPageSize * (first + pp0 + lane);  // position of the page's first key
            PageMeta m;
            m.ks = ok ? ks * kUp24 : 0.f;
            m.vs = ok ? vs : 0.f;
            m.nv = ok ? min(kPageSize, L - key0) : 0;
            m.lo = kWindow ? max(0, L - a.window - key0) : 0;  // keys before the sliding window are hidden
            wmeta[stage * U + lane] = m;
        }
        const uint32_t oks = __ballot_sync(0xffffffffu, ok);
        __syncwarp();  // the pages' metadata before the arrival
        uint64_t *bar = &wbar[stage];
        if (lane == 0) {
            wunit[stage] = UnitMeta{c.b, c.g, flags};
            if (oks)
                mbar_arrive_expect_tx(bar, __popc(oks) * 2 * C::kPageBytes);
            else
                mbar_arrive(bar);
        }
        __syncwarp();
        if (ok) {
            uint8_t *kb = wbuf + stage * C::kStageBytes + lane * C::kPageBytes;
            tma_load_4d_hint(kb, &kmap, bar, 0, 0, c.g, pg, policy);
            tma_load_4d_hint(kb + U * C::kPageBytes, &vmap, bar, 0, 0, c.g, pg, policy);
        }
    };

#pragma unroll 1
    for (int st = 0; st < S; ++st) produce(st);

    const int gr = lane >> 2, t4 = lane & 3;
    // K: this lane's MMA rows are tokens gr and gr + 8; its bytes are [t4 * D/4, +D/4)
    uint32_t koff[2][C::kKWords / 4];
#pragma unroll
    for (int i = 0; i < C::kKWords / 4; ++i) {
        koff[0][i] = page_off<D>(gr, t4 * (D / 4) + 16 * i);
        koff[1][i] = page_off<D>(gr + 8, t4 * (D / 4) + 16 * i);
    }
    // V: the lane's row address of the transposing loads, 16 bytes of a token each: matrices 0 and 1
    // are tokens 0-7 and 8-15 of one 16-byte column block, 2 and 3 of the next
    uint32_t voff[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) voff[i] = page_off<D>(lane & 15, 16 * (2 * i + (lane >> 4)));

    uint32_t qf[C::kKSteps][NH][2];
    float acc[C::kMTiles][NH][4];
    float mr[NH][2], ls[NH][2];
    float qoff[NH][2];                // -128 * 2^-24 * sum of q, per head
    float f0 = 0.f;                   // score factor but for the page's scale and 2^24
    float v_top = 0.f, v_inv = 0.f;   // 2^E and 2^-E

    for (int u = 0; u < n_units; ++u) {
        const int stage = u % S;
        if (!__all_sync(0xffffffffu, mbar_wait_sleep(&wbar[stage], (uint32_t)((u / S) & 1), a.wait_limit_ns))) {
            // give up (all lanes together: the outcome is voted): record it, let the copies
            // already issued land, leave
            if (lane == 0) set_status(a.status, SINKATTN_STATUS_WAIT_TIMEOUT);
            for (int v = u; v < produced; ++v)
                mbar_wait(&wbar[v % S], (uint32_t)((v / S) & 1), kDrainLimitNs);
            return;
        }
        const UnitMeta cur = wunit[stage];
        if (cur.flags & kStart) {
            const __nv_bfloat16 *qg = reinterpret_cast<const __nv_bfloat16 *>(a.q) +
                                      ((int64_t)cur.b * a.Hq + (int64_t)cur.g * a.G) * D;
            uint32_t mx = 0;  // the largest finite |q| of the lane, as bf16 bits
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                const int h = nt * 8 + gr;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {  // 8 bf16 per 16-byte load
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (h < a.G)
                        w = *reinterpret_cast<const uint4 *>(qg + h * D + t4 * (D / 4) + 8 * i);
                    // elements 8i .. 8i+7 of the lane's run: k-steps 2i and 2i + 1
                    qf[2 * i][nt][0] = w.x;
                    qf[2 * i][nt][1] = w.y;
                    qf[2 * i + 1][nt][0] = w.z;
                    qf[2 * i + 1][nt][1] = w.w;
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = x[e] & 0x7FFFu, hi = (x[e] >> 16) & 0x7FFFu;
                        mx = max(mx, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                    }
                }
            }
            // q times 2^(14 - e), e the exponent of the group's largest entry (kept where both
            // powers are normal floats), with the sign of the score scale
            const int ex = min(max((int)(__reduce_max_sync(0xffffffffu, mx) >> 7), 20), 254);
            const float down = copysignf(__uint_as_float((uint32_t)(268 - ex) << 23), a.scale_log2);
            f0 = fabsf(a.scale_log2) * __uint_as_float((uint32_t)(ex - 14) << 23);
#pragma unroll
            for (int kk = 0; kk < C::kKSteps; ++kk)
#pragma unroll
                for (int nt = 0; nt < NH; ++nt) {
                    // (elements 0, 1) and (2, 3) to (0, 2) and (1, 3), the order of the codes' pairs
                    const uint32_t x = bf16x2_to_f16x2_times(qf[kk][nt][0], down);
                    const uint32_t y = bf16x2_to_f16x2_times(qf[kk][nt][1], down);
                    qf[kk][nt][0] = __byte_perm(x, y, 0x5410);
                    qf[kk][nt][1] = __byte_perm(x, y, 0x7632);
                }
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                float o[4] = {0.f, 0.f, 0.f, 0.f};  // every row the same: columns 2 t4 and 2 t4 + 1
#pragma unroll
                for (int kk = 0; kk < C::kKSteps; ++kk)
                    mma_f16_16816(o, kMinus128, kMinus128, kMinus128, kMinus128, qf[kk][nt][0], qf[kk][nt][1]);
                qoff[nt][0] = o[0];
                qoff[nt][1] = o[1];
            }
#pragma unroll
            for (int mt = 0; mt < C::kMTiles; ++mt)
#pragma unroll
                for (int nt = 0; nt < NH; ++nt)
                    acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                mr[nt][0] = mr[nt][1] = -INFINITY;
                ls[nt][0] = ls[nt][1] = 0.f;
            }
            v_top = v_inv = 0.f;
        }

        const uint8_t *kb = wbuf + stage * C::kStageBytes;  // K of page j at kb + j * kPageBytes
        const uint8_t *vb = kb + U * C::kPageBytes;         // V of page j at vb + j * kPageBytes
        int nv[U], klo[U];
        float2 psc[U];
        // S^T = K Q^T per page: rows tokens, columns heads
        float s[U][NH][4];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const PageMeta m = wmeta[stage * U + j];
            nv[j] = m.nv;
            klo[j] = kWindow ? m.lo : 0;
            psc[j] = make_float2(m.ks, m.vs);
            uint32_t kw[2][C::kKWords];  // K rows gr, gr + 8: the lane's run of D/4 bytes
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < C::kKWords / 4; ++i) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(kb + j * C::kPageBytes + koff[r][i]);
                    kw[r][4 * i] = w.x;
                    kw[r][4 * i + 1] = w.y;
                    kw[r][4 * i + 2] = w.z;
                    kw[r][4 * i + 3] = w.w;
                }
#pragma unroll
            for (int kk = 0; kk < C::kKSteps; ++kk) {
                const uint32_t a0 = sub_even(kw[0][kk]), a2 = sub_odd(kw[0][kk]);
                const uint32_t a1 = sub_even(kw[1][kk]), a3 = sub_odd(kw[1][kk]);
#pragma unroll
                for (int nt = 0; nt < NH; ++nt) {
                    if (kk == 0)
                        mma_f16_16816_from(s[j][nt], qoff[nt][0], qoff[nt][1], a0, a1, a2, a3, qf[0][nt][0], qf[0][nt][1]);
                    else
                        mma_f16_16816(s[j][nt], a0, a1, a2, a3, qf[kk][nt][0], qf[kk][nt][1]);
                }
            }
        }
        // V of a page, by transposing loads of its byte pairs: v[mt][0] the pairs (16mt + 2gr, + 1) of
        // tokens 2 t4 and 2 t4 + 1, v[mt][1] of the tokens 8 further
        auto load_v = [&](int j, uint32_t (&v)[C::kMTiles][2]) {
            const uint32_t base = smem_u32(vb) + j * C::kPageBytes;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                ldsm_x4_t(base + voff[i], v[2 * i][0], v[2 * i][1], v[2 * i + 1][0], v[2 * i + 1][1]);
        };
        // The unit's V goes into registers and the stage back at once, so that the next copy overlaps
        // the rest of this unit's arithmetic.
        uint32_t vw[U][C::kMTiles][2];
#pragma unroll
        for (int j = 0; j < U; ++j) load_v(j, vw[j]);
        fence_proxy_async_smem();
        __syncwarp();
        produce(stage);

        // scores, hidden keys at -inf (every page but a sequence's last, and a window's first, is whole)
        bool raise = false;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float f = f0 * psc[j].x;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                s[j][nt][0] *= f;
                s[j][nt][1] *= f;
                s[j][nt][2] *= f;
                s[j][nt][3] *= f;
            }
            if (nv[j] < kPageSize || (kWindow && klo[j] > 0)) {  // warp-uniform
                const bool ok0 = gr < nv[j] && gr >= klo[j], ok1 = gr + 8 < nv[j] && gr + 8 >= klo[j];
#pragma unroll
                for (int nt = 0; nt < NH; ++nt) {
                    s[j][nt][0] = ok0 ? s[j][nt][0] : -INFINITY;
                    s[j][nt][1] = ok0 ? s[j][nt][1] : -INFINITY;
                    s[j][nt][2] = ok1 ? s[j][nt][2] : -INFINITY;
                    s[j][nt][3] = ok1 ? s[j][nt][3] : -INFINITY;
                }
            }
        }
        float cm[NH][2];  // the lane's maximum per column
#pragma unroll
        for (int nt = 0; nt < NH; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                cm[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
                for (int j = 1; j < U; ++j) cm[nt][e] = fmax3(cm[nt][e], s[j][nt][e], s[j][nt][2 + e]);
                raise |= cm[nt][e] > mr[nt][e] + kMaxSlack;
            }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = col_max(cm[nt][e]);
                    const float mn = x > mr[nt][e] + kMaxSlack ? x : mr[nt][e];
                    const float al = mr[nt][e] == -INFINITY ? 0.f : fast_exp2(mr[nt][e] - mn);
                    mr[nt][e] = mn;
                    ls[nt][e] *= al;
#pragma unroll
                    for (int mt = 0; mt < C::kMTiles; ++mt) {
                        acc[mt][nt][e] *= al;
                        acc[mt][nt][2 + e] *= al;
                    }
                }
        }
        // a V scale above every one so far: O^T to the next power of two, exactly
        float vmx = psc[0].y;
#pragma unroll
        for (int j = 1; j < U; ++j) vmx = fmaxf(vmx, psc[j].y);
        if (vmx > v_top) {  // warp-uniform
            const float top = __uint_as_float((__float_as_uint(vmx) + 0x7FFFFFu) & 0x7F800000u);
            const float inv = 1.0f / top, move = v_top * inv;
#pragma unroll
            for (int mt = 0; mt < C::kMTiles; ++mt)
#pragma unroll
                for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[mt][nt][i] *= move;
            v_top = top;
            v_inv = inv;
        }
        uint32_t pb[U][NH][2];
#pragma unroll
        for (int nt = 0; nt < NH; ++nt) {
            const float r0 = mr[nt][0] == -INFINITY ? 0.f : mr[nt][0] - kPShift;
            const float r1 = mr[nt][1] == -INFINITY ? 0.f : mr[nt][1] - kPShift;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const float w = psc[j].y * v_inv;
                const float p0 = fast_exp2(s[j][nt][0] - r0), p1 = fast_exp2(s[j][nt][1] - r1);
                const float p2 = fast_exp2(s[j][nt][2] - r0), p3 = fast_exp2(s[j][nt][3] - r1);
                ls[nt][0] += p0 + p2;
                ls[nt][1] += p1 + p3;
                // P^T fragments: transpose (token, head) blocks to (head, token)
                pb[j][nt][0] = movmatrix_t(pack_f16x2(p0 * w, p1 * w));
                pb[j][nt][1] = movmatrix_t(pack_f16x2(p2 * w, p3 * w));
            }
        }

        // O^T += V^T P^T, one 16-token k-step per page; first what the offset codes will add too much
#pragma unroll
        for (int nt = 0; nt < NH; ++nt) {
            float o[4];
            mma_f16_16816_from(o, 0.f, 0.f, kMinus128, kMinus128, kMinus128, kMinus128, pb[0][nt][0], pb[0][nt][1]);
#pragma unroll
            for (int j = 1; j < U; ++j)
                mma_f16_16816(o, kMinus128, kMinus128, kMinus128, kMinus128, pb[j][nt][0], pb[j][nt][1]);
            const float2 off = make_float2(o[0], o[1]);
#pragma unroll
            for (int mt = 0; mt < C::kMTiles; ++mt) {
                const float2 x = fadd2(make_float2(acc[mt][nt][0], acc[mt][nt][1]), off);
                const float2 y = fadd2(make_float2(acc[mt][nt][2], acc[mt][nt][3]), off);
                acc[mt][nt][0] = x.x;
                acc[mt][nt][1] = x.y;
                acc[mt][nt][2] = y.x;
                acc[mt][nt][3] = y.y;
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            // rows 0-7 of m-tile mt are head_dim 16mt + 2gr, rows 8-15 the odd ones beside them
#pragma unroll
            for (int mt = 0; mt < C::kMTiles; ++mt) {
                const uint32_t a0 = sub_even(vw[j][mt][0]), a1 = sub_odd(vw[j][mt][0]);
                const uint32_t a2 = sub_even(vw[j][mt][1]), a3 = sub_odd(vw[j][mt][1]);
#pragma unroll
                for (int nt = 0; nt < NH; ++nt)
                    mma_f16_16816(acc[mt][nt], a0, a1, a2, a3, pb[j][nt][0], pb[j][nt][1]);
            }
        }

        if (cur.flags & kEnd) {
            const bool whole = cur.flags & kWhole;
            const int64_t slot = (int64_t)wglob + (int64_t)cur.b * a.Hkv + cur.g;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float L = col_sum(ls[nt][e]);
                    const int hc = nt * 8 + 2 * t4 + e;  // column (head in the group)
                    // reference of the state: probabilities were taken against mr - kPShift
                    const float m = mr[nt][e] == -INFINITY ? -INFINITY : mr[nt][e] - kPShift;
                    if (hc >= a.G) continue;
                    const int h = cur.g * a.G + hc;
                    if (whole) {
                        const float sk = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
                        const float M = fmaxf(m, sk);
                        float scl = 0.f, lse2 = -INFINITY;
                        if (M != -INFINITY) {
                            const float wm = m == -INFINITY ? 0.f : exp2f(m - M);
                            const float den = L * wm + (sk == -INFINITY ? 0.f : exp2f(sk - M));
                            scl = wm / den;
                            lse2 = M + log2f(den);
                        }
                        __nv_bfloat16 *og = reinterpret_cast<__nv_bfloat16 *>(a.out) +
                                            ((int64_t)cur.b * a.Hq + h) * D + 2 * gr;
#pragma unroll
                        for (int mt = 0; mt < C::kMTiles; ++mt)
                            *reinterpret_cast<uint32_t *>(og + 16 * mt) = pack_bf16x2(
                                acc[mt][nt][e] * kUp24 * scl * v_top, acc[mt][nt][2 + e] * kUp24 * scl * v_top);
                        if (a.lse && gr == 0) a.lse[(int64_t)cur.b * a.Hq + h] = lse2 * kLn2;
                    } else {
                        const int64_t row = slot * a.G + hc;
                        constexpr float kUp = kUp24 * kStateDown;
                        float *pa = a.part_acc + row * D + 2 * gr;
#pragma unroll
                        for (int mt = 0; mt < C::kMTiles; ++mt)
                            *reinterpret_cast<float2 *>(pa + 16 * mt) =
                                make_float2(acc[mt][nt][e] * kUp * v_top, acc[mt][nt][2 + e] * kUp * v_top);
                        if (gr == 0)
                            *reinterpret_cast<float2 *>(a.part_ml + row * 2) =
                                make_float2(m + kPShift + kMaxSlack, L * kStateDown);
                    }
                }
        }
    }
    // Near the end of the grid the merge may take its place on the SMs; it waits for this grid before
    // it reads.  (Not earlier: its waiting blocks would hold the threads of the SMs that max_sms
    // keeps free for others.)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Log-sum-exp merge of the partial states of one (sequence, query head), the sink counted once.
// A block of 128 threads: D/4 threads span the head's outputs, the others split the states (8 ways
// at head_dim 64, 4 at 128), so that the loads of many states are in flight at once; each part
// keeps its own maximum, and the parts meet in shared memory in a fixed order.  It is launched as
// a programmatic dependent of the split-KV kernel: its blocks are set up while that one ends (one
// sequence of 4097 tokens: 10.5 us for both kernels).
template <int D>
__global__ void __launch_bounds__(128) merge_int8_kernel(const DecodeArgs a) {
    constexpr int kQuads = D / 4, kParts = 128 / kQuads;
    __shared__ float4 s_o[kParts][kQuads];
    __shared__ float2 s_ml[kParts];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, g = h / a.G, r = h % a.G;
    const int d4 = threadIdx.x % kQuads, part = threadIdx.x / kQuads;
    const int p0 = a.ws_prefix[b], pb = a.ws_prefix[b + 1] - p0;
    const int64_t row = (int64_t)b * a.Hq + h;
    __nv_bfloat16 *og = reinterpret_cast<__nv_bfloat16 *>(a.out) + row * D + d4 * 4;
    if (pb == 0) {
        if (part == 0) *reinterpret_cast<uint2 *>(og) = make_uint2(0u, 0u);
        if (threadIdx.x == 0 && a.lse) a.lse[row] = a.sinks ? a.sinks[h] : -INFINITY;
        return;
    }
    const int64_t start = (int64_t)a.Hkv * p0 + (int64_t)g * pb, last = start + pb - 1;
    const int64_t per = a.ws_plan[1];
    const int64_t w_lo = start / per, w_hi = last / per;
    if (w_lo == w_hi) return;  // finished by the split-KV kernel
    const int nsplit = (int)(w_hi - w_lo + 1);
    const int64_t slot0 = w_lo + (int64_t)b * a.Hkv + g;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = part; s < nsplit; s += kParts) m = fmaxf(m, a.part_ml[((slot0 + s) * a.G + r) * 2]);
    if (m != -INFINITY) {
#pragma unroll 4
        for (int s = part; s < nsplit; s += kParts) {
            const int64_t at = (slot0 + s) * a.G + r;
            const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + at * 2);
            const float4 v = *reinterpret_cast<const float4 *>(a.part_acc + at * D + d4 * 4);
            const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
            l = fmaf(ml.y, w, l);
            o.x = fmaf(v.x, w, o.x);
            o.y = fmaf(v.y, w, o.y);
            o.z = fmaf(v.z, w, o.z);
            o.w = fmaf(v.w, w, o.w);
        }
    }
    s_o[part][d4] = o;
    if (d4 == 0) s_ml[part] = make_float2(m, l);
    __syncthreads();
    if (part > 0) return;
    const float sk = a.sinks ? a.sinks[h] * kLog2e : -INFINITY;
    float M = sk;
#pragma unroll
    for (int i = 0; i < kParts; ++i) M = fmaxf(M, s_ml[i].x);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float lse2 = -INFINITY;
    if (M != -INFINITY) {
        float den = sk == -INFINITY ? 0.f : exp2f(sk - M);
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const float2 ml = s_ml[i];
            const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
            const float4 v = s_o[i][d4];
            den = fmaf(ml.y, w, den);
            sum.x = fmaf(v.x, w, sum.x);
            sum.y = fmaf(v.y, w, sum.y);
            sum.z = fmaf(v.z, w, sum.z);
            sum.w = fmaf(v.w, w, sum.w);
        }
        const float inv = 1.f / den;
        sum.x *= inv;
        sum.y *= inv;
        sum.z *= inv;
        sum.w *= inv;
        lse2 = M + log2f(den);
    }
    *reinterpret_cast<uint2 *>(og) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
    if (d4 == 0 && a.lse) a.lse[row] = lse2 * kLn2;
}

template <int D, int NH>
cudaError_t int8_shape_for(int B, int device, int *ctas, int *warps, int *smem) {
    using C = Int8Cfg<D, NH>;
    const int bytes = int8_smem_bytes<D, NH>(B);
    int optin = 0, sms = 0, occ = 1 << 30;
    cudaError_t e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return e;
    const void *kernels[2] = {reinterpret_cast<const void *>(decode_int8_kernel<D, NH, false>),
                              reinterpret_cast<const void *>(decode_int8_kernel<D, NH, true>)};
    for (const void *k : kernels) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, k);
        if (e != cudaSuccess) return e;
        const int ceiling = optin - (int)fa.sharedSizeBytes;
        if (bytes > ceiling) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ceiling);
        if (e != cudaSuccess) return e;
        int o = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, k, C::kThreads, bytes);
        if (e != cudaSuccess) return e;
        occ = min(occ, o);
    }
    if (occ < 1) return cudaErrorInvalidConfiguration;
    *ctas = sms * occ;
    *warps = C::kWarps;
    *smem = bytes;
    return cudaSuccess;
}

}  // namespace

cudaError_t decode_int8_launch_shape(int D, int G, int B, int device, int *ctas, int *warps_per_cta,
                                     int *smem_bytes) {
    struct Entry {
        int device, D, NH, B, ctas, warps, smem;
    };
    static std::mutex mu;
    static std::vector<Entry> cache;
    const int NH = G > 8 ? 2 : 1;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (const Entry &e : cache)
            if (e.device == device && e.D == D && e.NH == NH && e.B == B) {
                *ctas = e.ctas;
                *warps_per_cta = e.warps;
                *smem_bytes = e.smem;
                return cudaSuccess;
            }
    }
    cudaError_t e;
    if (D == 64 && NH == 1)
        e = int8_shape_for<64, 1>(B, device, ctas, warps_per_cta, smem_bytes);
    else if (D == 64)
        e = int8_shape_for<64, 2>(B, device, ctas, warps_per_cta, smem_bytes);
    else if (D == 128 && NH == 1)
        e = int8_shape_for<128, 1>(B, device, ctas, warps_per_cta, smem_bytes);
    else if (D == 128)
        e = int8_shape_for<128, 2>(B, device, ctas, warps_per_cta, smem_bytes);
    else
        return cudaErrorInvalidValue;
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> lock(mu);
        if (cache.size() > 256) cache.clear();
        cache.push_back({device, D, NH, B, *ctas, *warps_per_cta, *smem_bytes});
    }
    return e;
}

cudaError_t launch_decode_int8(int D, const DecodeArgs &a, const CUtensorMap &kmap, const CUtensorMap &vmap,
                               int ctas, int smem_bytes, cudaStream_t stream) {
    const bool w = a.window > 0, two = a.G > 8;
#define SINKATTN_INT8_LAUNCH(DD, NN, WW) \
    decode_int8_kernel<DD, NN, WW><<<ctas, Int8Cfg<DD, NN>::kThreads, smem_bytes, stream>>>(kmap, vmap, a)
    if (D == 64) {
        if (two) {
            if (w) SINKATTN_INT8_LAUNCH(64, 2, true); else SINKATTN_INT8_LAUNCH(64, 2, false);
        } else {
            if (w) SINKATTN_INT8_LAUNCH(64, 1, true); else SINKATTN_INT8_LAUNCH(64, 1, false);
        }
    } else {
        if (two) {
            if (w) SINKATTN_INT8_LAUNCH(128, 2, true); else SINKATTN_INT8_LAUNCH(128, 2, false);
        } else {
            if (w) SINKATTN_INT8_LAUNCH(128, 1, true); else SINKATTN_INT8_LAUNCH(128, 1, false);
        }
    }
#undef SINKATTN_INT8_LAUNCH
    return cudaGetLastError();
}

cudaError_t launch_merge_int8(int D, const DecodeArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.B * (unsigned)a.Hq);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 64 ? cudaLaunchKernelEx(&cfg, merge_int8_kernel<64>, a)
                   : cudaLaunchKernelEx(&cfg, merge_int8_kernel<128>, a);
}

}  // namespace sinkattn
