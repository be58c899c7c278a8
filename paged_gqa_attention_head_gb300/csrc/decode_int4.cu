// Split-KV paged decode with per-head sinks over a 4-bit cache (append_int4.cu): value = s (code - z)
// with a scale s and a zero code z for every token and 32 channels.
//
// The plan is that of the INT8 decode: every warp takes an equal run of units of pages, the products
// run on m16n8k16 f16 MMAs with online softmax, and a merge joins the split sequences' states.  A
// page's K and V of a head are one contiguous record of 18 D bytes, copied by one untiled bulk copy.
// What four bits change is the arithmetic that a byte of the cache brings (ALU instructions issue every
// other cycle, an MMA takes the tensor cores 8 cycles and the ALU some 4 beside them), so that is what
// the layout and the kernel save on:
//   * a code is taken as the f16 subnormal code * 2^-24: a 32-bit word of eight codes becomes operand
//     registers by ANDs alone.  The odd codes of a byte stay four bits up: for K 16 times their value,
//     against a sixteenth of the query's entries; for V together with the even one beside it (one AND
//     less), which the output rows are parted from at the end;
//   * K's contraction runs over channels in the word's order, which is the query's too; V comes by
//     transposing 8x8 loads of 16-bit elements, four channels of a token: a register holds the same four
//     channels of two neighbouring tokens, and the ANDs part the channels;
//   * the words of a page come by 8x8 loads whose eight row addresses are the same: plain, a lane gets
//     the words of its two neighbouring tokens; transposed, its own token's word twice (the scale as
//     a float: one AND; z as an f16 pair: another);
//   * z comes off the codes, exactly, by one f16 multiplication and addition for two of them.  (Off the
//     products - z times -sum of the group's q, and z times P, as MMAs of their own - the batch below takes 160
//     us where this takes 165, but the sums that cancel leave the scores of single keys 4e-6 off, ten times
//     as much as this);
//   * a group's K scores are multiplied by s in fp32; P of a group is taken times s, relative to the
//     power of two above the largest V scale met, and rounded once to f16, as in the INT8 decode.
// Groups of up to 8 heads: S^T = K Q^T and O^T = V^T P^T, tokens and channels on the M axis, heads on N,
// with P transposed between them.  16 heads fill the M axis themselves: S = Q K^T and O = P V, P in place.
// The running maximum moves only when a score passes it by more than 8 (log2).
// FP8 MMAs (a code as the E4M3 subnormal code * 2^-9, half the ANDs, q in three E5M2 parts) are made of
// conversions and f16 MMAs here: 226 us.
// Measured: 64 sequences up to 131072 tokens, 64/8 heads of 64 (0.71 GB) 165 us, 4.3 TB/s; 64 sequences up to
// 16384, 64/4 heads of 128 (0.31 GB) 97 us, 3.2 TB/s.  Each instruction added to the first shows (an AND 2.0
// cycles a page and scheduler, an MMA 6, an f16 multiplication and addition 1.4, of ~275): it is bound by
// their issue.  The second is bound by the latencies of the two warps a scheduler that its registers allow.
#include <math.h>

#include <mutex>
#include <vector>

#include "decode_common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace sinkattn {

namespace {

template <int D, int NH>
struct Int4Cfg {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = kWarps * 32;
    // Pages of a unit, one copy stage: what a unit costs beside its pages' arithmetic is ~100 instructions, so as
    // many as two stages for each warp leave room for (head_dim 64: 4 pages 176 us where 8 take 165; 128 and 16
    // heads, whose registers allow two CTAs an SM: 4 pages 99.9 us, 6 96.8).
    static constexpr int kPPU = D == 64 ? 8 : NH == 1 ? 4 : 6;
    // Pages whose scores are held at once: what a step costs beside them, against registers and the time of a
    // short sequence (head_dim 64: 2 pages 167 us, 4 165, 8 164, where one sequence of 4097 tokens takes 9.8, 10.3 and
    // 10.7; 128 and 16 heads: 1 page 101 us, 2 96.8, 3 97.4).
    static constexpr int kStep = D == 64 && NH == 1 ? 4 : 2;
    static_assert(kPPU % kStep == 0, "a step stays inside its unit");
    static constexpr int kStages = 2;
    static constexpr int kRec = 9 * D;                         // K (or V) of a (page, head)
    static constexpr int kPageBytes = 2 * kRec;
    static constexpr int kStageBytes = kPPU * kPageBytes;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kGroups = D / 32;
    static constexpr int kCtas = NH == 2 && D == 128 ? 2 : 3;  // CTAs an SM, by registers
};

constexpr float kMaxSlack = 8.f;  // the running maximum, a whole number, moves when a score passes it by more
constexpr float kPUp = 128.f;     // P = 2^(s - m), at most 2^8, enters its product 2^7 times as large: f16's range
constexpr float kStateDown = 1.f / 256.f;  // states leave with their sums over 2^kMaxSlack, the largest P
constexpr float kUp24 = 16777216.f;          // 2^24
constexpr float kScaleLeast = 7.888609052210118e-31f;  // 2^-100, the least V scale that P is taken relative to
constexpr uint32_t kEven = 0x000F000Fu, kOdd = 0x00F000F0u;  // pairs of codes in place, and 16 times them
constexpr uint32_t kBoth = 0x00FF00FFu;                      // pairs of (even code + 16 odd code)

// Scale of the word in the upper or the lower half of a pair.
__device__ __forceinline__ float scale_hi(uint32_t w) { return __uint_as_float(w & 0xFFF00000u); }
__device__ __forceinline__ float scale_lo(uint32_t w) { return __uint_as_float((w << 16) & 0xFFF00000u); }
// Over the four lanes that share lane >> 2.
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// Bytes 1 and 3 of a word as a pair.
__device__ __forceinline__ uint32_t high_bytes(uint32_t w) { return __byte_perm(w, 0u, 0x4341); }
// x + z * m in f16 pairs (exact here: multiples of 2^-24 below 2^-16).
__device__ __forceinline__ uint32_t fma_h2(uint32_t z, uint32_t m, uint32_t x) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(z), "r"(m), "r"(x));
    return r;
}
// The codes of a word less z: pairs in place [0], [2] and 16 times their value [1], [3], of the lower and the
// upper bytes.
__device__ __forceinline__ void less_z(uint32_t (&c)[4], uint32_t w, uint32_t z) {
    constexpr uint32_t m1 = 0xBC00BC00u, m16 = 0xCC00CC00u;  // -1, -16
    const uint32_t h = w >> 8;
    c[0] = fma_h2(z, m1, w & kEven);
    c[1] = fma_h2(z, m16, w & kOdd);
    c[2] = fma_h2(z, m1, h & kEven);
    c[3] = fma_h2(z, m16, h & kOdd);
}

// What the arithmetic needs of a unit.
struct __align__(16) UnitMeta4 {
    int b, g;     // sequence, KV head
    int flags;    // kStart | kEnd | kWhole
    int pages;    // bit j: page j is there
    int end, lo;  // its tokens lo .. end - 1, counted from its first page's first, are visible
    int pad[2];
};
constexpr int kStart = 1, kEnd = 2, kWhole = 4;  // first / last unit of a segment; the segment is all of (b, g)

template <int D, int NH>
int int4_smem_bytes(int B) {
    using C = Int4Cfg<D, NH>;
    return 128 /* alignment slack */ + C::kWarps * C::kWarpBytes + C::kWarps * C::kStages * (8 + (int)sizeof(UnitMeta4)) +
           (B + 1) * 4;
}

// Length of a sequence, held to what its block table can name.
__device__ __forceinline__ int length_of(const DecodeArgs &a, int b) {
    return (int)min((int64_t)max(a.seq_lens[b], 0), (int64_t)a.max_pages * kPageSize);
}
template <bool kWindow>
__device__ __forceinline__ int first_page(const DecodeArgs &a, int L) {
    return kWindow && L > a.window ? (L - a.window) / kPageSize : 0;
}

// Exclusive prefix sum of the sequences' units (kPPU visible pages each), into shared memory.
template <int kPPU, bool kWindow>
__device__ void scan_units(const DecodeArgs &a, int *s_prefix) {
    __shared__ int s_warp_tot[4];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int per_t = (a.B + 127) / 128;
    const int b0 = min(a.B, tid * per_t), b1 = min(a.B, b0 + per_t);
    int local = 0;
    for (int b = b0; b < b1; ++b) {
        const int raw = a.seq_lens[b], L = length_of(a, b);
        if (raw != L) set_status(a.status, SINKATTN_STATUS_BAD_LENGTH);
        const int n = ((L + kPageSize - 1) / kPageSize - first_page<kWindow>(a, L) + kPPU - 1) / kPPU;
        s_prefix[b] = n;
        local += n;
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp_tot[wid] = incl;
    __syncthreads();
    int run = incl - local;
    for (int w = 0; w < wid; ++w) run += s_warp_tot[w];
    for (int b = b0; b < b1; ++b) {
        const int n = s_prefix[b];
        s_prefix[b] = run;
        run += n;
    }
    if (tid == 0) s_prefix[a.B] = s_warp_tot[0] + s_warp_tot[1] + s_warp_tot[2] + s_warp_tot[3];
    __syncthreads();
}

// NH: 8-head tiles of the query group (1 for G <= 8, 2 for G = 16).
template <int D, int NH, bool kWindow>
__global__ void __launch_bounds__(Int4Cfg<D, NH>::kThreads, Int4Cfg<D, NH>::kCtas) decode_int4_kernel(const DecodeArgs a) {
    using C = Int4Cfg<D, NH>;
    constexpr int S = C::kStages, U = C::kPPU, W = C::kStep, NG = C::kGroups;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    UnitMeta4 *s_unit = reinterpret_cast<UnitMeta4 *>(smem + C::kWarps * C::kWarpBytes);  // [warp][stage]
    uint64_t *bars = reinterpret_cast<uint64_t *>(s_unit + C::kWarps * S);
    int *s_prefix = reinterpret_cast<int *>(bars + C::kWarps * S);

    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (lane < S) mbar_init(&bars[wid * S + lane], 1);
    fence_mbar_init();
    scan_units<U, kWindow>(a, s_prefix);  // contains __syncthreads

    const int64_t T = (int64_t)a.Hkv * s_prefix[a.B];
    const int64_t per = (T + a.total_warps - 1) / a.total_warps;
    if (blockIdx.x == 0) {
        for (int b = tid; b <= a.B; b += blockDim.x) a.ws_prefix[b] = s_prefix[b];
        if (tid == 0) {
            a.ws_plan[0] = T;
            a.ws_plan[1] = per > 0 ? per : 1;
        }
    }
    const int wglob = blockIdx.x * C::kWarps + wid;
    const int64_t u_begin = (int64_t)wglob * per;
    if (u_begin >= T) return;  // warp-uniform; no block-wide barrier follows
    const int n_units = (int)min(per, T - u_begin);

    uint8_t *wbuf = smem + wid * C::kWarpBytes;
    uint64_t *wbar = bars + wid * S;
    UnitMeta4 *wunit = s_unit + wid * S;

    // The copy side: its unit's sequence, KV head and place in the list (pb units in all), the first unit
    // of its segment and the units copied so far; and what follows from the sequence: its length, the
    // first visible page, the visible pages and its row of the block table from there.
    int b, g, p, pb, p_seg0, produced = 0;
    {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)a.Hkv * s_prefix[mid] <= u_begin)
                lo = mid;
            else
                hi = mid - 1;
        }
        b = lo;
        pb = s_prefix[lo + 1] - s_prefix[lo];
        const int local = (int)(u_begin - (int64_t)a.Hkv * s_prefix[lo]);
        g = local / pb;
        p = p_seg0 = local % pb;
    }
    int L, first, npv;
    const int32_t *row;
    // Lane l holds the row's entry of visible page win + l (-1 past the last); those of the next window of
    // kWin pages, whole units, are loaded with it.
    constexpr int kWin = 32 / U * U;
    int win, win_val, nxt_val;
    auto entry = [&](int q) { return q < npv ? row[q] : -1; };
    auto sequence = [&](int at) {
        L = length_of(a, b);
        first = first_page<kWindow>(a, L);
        npv = (L + kPageSize - 1) / kPageSize - first;
        row = a.block_table + (int64_t)b * a.max_pages + first;
        win = at - at % kWin;
        win_val = entry(win + lane);
        nxt_val = entry(win + kWin + lane);
    };
    sequence(p * U);
    const uint64_t policy = l2_policy_evict_first();
    // The next unit, if there is one, into a stage: lanes 0 .. U - 1 take a page each.
    auto produce = [&](int stage) {
        if (produced == n_units) return;
        ++produced;
        const int pp0 = p * U;
        if (pp0 >= win + kWin) {  // warp-uniform
            win += kWin;
            win_val = nxt_val;
            nxt_val = entry(win + kWin + lane);
        }
        const int pg = __shfl_sync(0xffffffffu, win_val, (pp0 - win + lane) & 31);
        const bool in = lane < U && pp0 + lane < npv, ok = in && (uint32_t)pg < (uint32_t)a.num_pages;
        const uint32_t oks = __ballot_sync(0xffffffffu, ok);
        uint64_t *bar = &wbar[stage];
        const bool last = p == pb - 1;
        if (lane == 0) {
            const int flags = (p == p_seg0 ? kStart : 0) | (last || produced == n_units ? kEnd : 0) |
                              (last && p_seg0 == 0 ? kWhole : 0);
            const int key0 = kPageSize * (first + pp0);  // position of the unit's first key
            UnitMeta4 &m = wunit[stage];
            *reinterpret_cast<int4 *>(&m.b) = make_int4(b, g, flags, (int)oks);
            *reinterpret_cast<int2 *>(&m.end) = make_int2(L - key0, kWindow ? L - a.window - key0 : 0);
            mbar_arrive_expect_tx(bar, __popc(oks) * C::kPageBytes);
        }
        __syncwarp();
        if (ok)
            bulk_load_hint(wbuf + stage * C::kStageBytes + lane * C::kPageBytes,
                           static_cast<const uint8_t *>(a.kv_int4) + ((int64_t)pg * a.Hkv + g) * C::kPageBytes,
                           C::kPageBytes, bar, policy);
        else if (in)
            set_status(a.status, SINKATTN_STATUS_BAD_PAGE);
        ++p;
        if (last) {
            p = p_seg0 = 0;
            if (++g == a.Hkv) {
                g = 0;
                do {
                    ++b;
                    pb = b < a.B ? s_prefix[b + 1] - s_prefix[b] : 1;
                } while (b < a.B && pb == 0);
                if (b < a.B) sequence(0);
            } else if (win != 0) {
                win = 0;
                win_val = entry(lane);
                nxt_val = entry(kWin + lane);
            }
        }
    };

#pragma unroll 1
    for (int st = 0; st < S; ++st) produce(st);

    const int gr = lane >> 2, t4 = lane & 3;
    // q in the order of its MMA operand: [2 i + x][e NH + nt] of head 8 nt + gr, channels 32 i + 8 t4 + 4 x + (0, 1)
    // (e 0) and a sixteenth of + (2, 3) (e 1)
    uint32_t qf[2 * NG][2 * NH];
    // O * 2^-24.  8 heads: [m-tile 2 i + x][.]: channels 32 i + 8 (gr / 2) + gr % 2 + 4 x (and of these plus 16
    // times the ones 2 further) of heads 2 t4, 2 t4 + 1; 16 heads: [4 i + n]: channels 32 i + 8 t4 + (0, 1) (n even)
    // + 2 n (and of those plus 16 times the ones 2 further, n odd) of heads gr, gr + 8
    float acc[2 * NG * NH][4];
    // of the lane's two heads (8: 2 t4, 2 t4 + 1; 16: gr, gr + 8): running maximum of the scores (log2), a score
    // above which (before its factor f0) it moves, -maximum (0 before the first key), sum of P
    float mr[2], thr[2], nr[2];
    float2 ls[NH];                    // 8 heads: of both; 16: of each, from even and from odd tokens
    float f0 = 0.f;                   // score factor
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
        const int4 cur = *reinterpret_cast<const int4 *>(&wunit[stage].b);  // b, g, flags, pages
        const int2 vis = *reinterpret_cast<const int2 *>(&wunit[stage].end);
        if (cur.z & kStart) {
            const __nv_bfloat16 *qg = reinterpret_cast<const __nv_bfloat16 *>(a.q) +
                                      ((int64_t)cur.x * a.Hq + (int64_t)cur.y * a.G) * D;
            uint32_t mx = 0;  // the largest finite |q| of the lane, as bf16 bits
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                const int h = nt * 8 + gr;
#pragma unroll
                for (int i = 0; i < NG; ++i) {  // channels 32 i + 8 t4 .. + 7
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (h < a.G) w = *reinterpret_cast<const uint4 *>(qg + h * D + 32 * i + 8 * t4);
                    qf[2 * i][nt] = w.x;
                    qf[2 * i][NH + nt] = w.y;
                    qf[2 * i + 1][nt] = w.z;
                    qf[2 * i + 1][NH + nt] = w.w;
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = x[e] & 0x7FFFu, hi = (x[e] >> 16) & 0x7FFFu;
                        mx = max(mx, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                    }
                }
            }
            // q times 2^(14 - e), e the exponent of the group's largest entry (kept where both powers are
            // normal floats), with the sign of the score scale
            const int ex = min(max((int)(__reduce_max_sync(0xffffffffu, mx) >> 7), 20), 254);
            const float down = copysignf(__uint_as_float((uint32_t)(268 - ex) << 23), a.scale_log2);
            // (never 0, so that a hidden key's -inf stays one)
            f0 = fmaxf(fabsf(a.scale_log2) * __uint_as_float((uint32_t)(ex - 14) << 23) * kUp24, 1e-37f);
#pragma unroll
            for (int kk = 0; kk < 2 * NG; ++kk)
#pragma unroll
                for (int e = 0; e < 2 * NH; ++e) {
                    const uint32_t w = qf[kk][e];
                    const float d = e >= NH ? down * 0.0625f : down;
                    qf[kk][e] = pack_f16x2(__uint_as_float(w << 16) * d, __uint_as_float(w & 0xFFFF0000u) * d);
                }
#pragma unroll
            for (int i = 0; i < 2 * NG * NH; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mr[e] = thr[e] = -INFINITY;
                nr[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < NH; ++e) ls[e] = make_float2(0.f, 0.f);
            v_top = v_inv = 0.f;
        }

        const uint32_t buf = smem_u32(wbuf + stage * C::kStageBytes);
#pragma unroll 1
        for (int j0 = 0; j0 < U; j0 += W) {
            if (vis.x <= kPageSize * j0) break;                               // warp-uniform: nothing left
            if (kWindow && vis.y >= kPageSize * (j0 + W)) continue;           // all of it before the window
            const uint32_t at = buf + j0 * C::kPageBytes;
            // some page of the step is missing, ragged or cut by the window
            const bool ragged = ((cur.w >> j0) & ((1 << W) - 1)) != (1 << W) - 1 || vis.x < kPageSize * (j0 + W) ||
                                (kWindow && vis.y > kPageSize * j0);
            // visible tokens of page j: lo(j) .. nv(j) - 1
            auto nv = [&](int j) { return (cur.w >> (j0 + j)) & 1 ? min(kPageSize, vis.x - kPageSize * (j0 + j)) : 0; };
            auto lo = [&](int j) { return kWindow ? vis.y - kPageSize * (j0 + j) : 0; };

            // Scores of the step's pages, a group's part times its tokens' scales, and the V scales.
            // 8 heads: [.][token half][token gr]: heads 2 t4, 2 t4 + 1.  16: [.][token half][head half]: tokens 2 t4 and + 1.
            float2 s[W][2][NH];
            float2 vs[W][NG][2];  // 8 heads: .x and .y of the lane's tokens gr, gr + 8 in [0]; 16: of its pairs of tokens
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const uint32_t kb = at + j * C::kPageBytes;
                uint32_t kc[NG][2], kw[NG][2], kz[NG][2], vw[NG][2];
#pragma unroll
                for (int i = 0; i < NG / 2; ++i) {
                    ldsm_x4(kb + 512 * i + 16 * lane, kc[2 * i][0], kc[2 * i][1], kc[2 * i + 1][0], kc[2 * i + 1][1]);
                    const uint32_t wa = kb + 8 * D + 64 * i + 16 * (lane >> 3);
                    if (NH == 1) {
                        ldsm_x4_t(wa, kw[2 * i][0], kw[2 * i][1], kw[2 * i + 1][0], kw[2 * i + 1][1]);
                        ldsm_x4_t(wa + C::kRec, vw[2 * i][0], vw[2 * i][1], vw[2 * i + 1][0], vw[2 * i + 1][1]);
                    } else {
                        ldsm_x4(wa, kw[2 * i][0], kw[2 * i][1], kw[2 * i + 1][0], kw[2 * i + 1][1]);
                        ldsm_x4_t(wa, kz[2 * i][0], kz[2 * i][1], kz[2 * i + 1][0], kz[2 * i + 1][1]);
                        ldsm_x4(wa + C::kRec, vw[2 * i][0], vw[2 * i][1], vw[2 * i + 1][0], vw[2 * i + 1][1]);
                    }
                }
                if (NH == 1) {
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        uint32_t c0[4], c1[4];
                        less_z(c0, kc[i][0], kw[i][0] & kEven);
                        less_z(c1, kc[i][1], kw[i][1] & kEven);
                        const float s0 = scale_hi(kw[i][0]), s1 = scale_hi(kw[i][1]);
                        float o[4];
                        mma_f16_16816_from(o, 0.f, 0.f, c0[0], c1[0], c0[1], c1[1], qf[2 * i][0], qf[2 * i][1]);
                        mma_f16_16816(o, c0[2], c1[2], c0[3], c1[3], qf[2 * i + 1][0], qf[2 * i + 1][1]);
                        // (one by one: a pair of one scale would be a move)
                        s[j][0][0].x = i ? fmaf(o[0], s0, s[j][0][0].x) : o[0] * s0;
                        s[j][0][0].y = i ? fmaf(o[1], s0, s[j][0][0].y) : o[1] * s0;
                        s[j][1][0].x = i ? fmaf(o[2], s1, s[j][1][0].x) : o[2] * s1;
                        s[j][1][0].y = i ? fmaf(o[3], s1, s[j][1][0].y) : o[3] * s1;
                        vs[j][i][0] = make_float2(scale_hi(vw[i][0]), scale_hi(vw[i][1]));
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < NG; ++i) {
                            const uint32_t(&x)[2 * NH] = qf[2 * i], (&y)[2 * NH] = qf[2 * i + 1];
                            uint32_t c[4];
                            less_z(c, kc[i][n], kz[i][n] & kEven);
                            float o[4];
                            mma_f16_16816_from(o, 0.f, 0.f, x[0], x[1], x[2 * NH - 2], x[2 * NH - 1], c[0], c[1]);
                            mma_f16_16816(o, y[0], y[1], y[2 * NH - 2], y[2 * NH - 1], c[2], c[3]);
                            const float2 sc = make_float2(scale_lo(kw[i][n]), scale_hi(kw[i][n]));
                            const float2 u = make_float2(o[0], o[1]), v = make_float2(o[2], o[3]);
                            s[j][n][0] = i ? ffma2(u, sc, s[j][n][0]) : fmul2(u, sc);
                            s[j][n][NH - 1] = i ? ffma2(v, sc, s[j][n][NH - 1]) : fmul2(v, sc);
                            vs[j][i][n] = make_float2(scale_lo(vw[i][n]), scale_hi(vw[i][n]));
                        }
                }
            }
            if (ragged) {  // hidden tokens: no score, and no scale, whatever lies there
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int n = nv(j), l = lo(j);
                    auto hidden = [&](int t) { return t >= n || t < l; };
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (NH == 1) {
                            if (!hidden(gr + 8 * r)) continue;
                            s[j][r][0] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
                            for (int i = 0; i < NG; ++i) (r ? vs[j][i][0].y : vs[j][i][0].x) = 0.f;
                        } else {
                            const bool x = hidden(2 * t4 + 8 * r), y = hidden(2 * t4 + 1 + 8 * r);
#pragma unroll
                            for (int e = 0; e < NH; ++e) {
                                if (x) s[j][r][e].x = -INFINITY;
                                if (y) s[j][r][e].y = -INFINITY;
                            }
#pragma unroll
                            for (int i = 0; i < NG; ++i) {
                                if (x) vs[j][i][r].x = 0.f;
                                if (y) vs[j][i][r].y = 0.f;
                            }
                        }
                    }
                }
            }
            // a score too far above the running maximum, or a V scale above every one so far
            float vmx = 0.f, cm[2];
#pragma unroll
            for (int j = 0; j < W; ++j) {
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int r = 0; r < NH; ++r) vmx = fmax3(vmx, vs[j][i][r].x, vs[j][i][r].y);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x[4];  // the lane's scores of its head e
                    if (NH == 1) {
                        x[0] = e ? s[j][0][0].y : s[j][0][0].x;
                        x[1] = e ? s[j][1][0].y : s[j][1][0].x;
                    } else {
                        x[0] = s[j][0][e * (NH - 1)].x, x[1] = s[j][0][e * (NH - 1)].y;
                        x[2] = s[j][1][e * (NH - 1)].x, x[3] = s[j][1][e * (NH - 1)].y;
                    }
                    cm[e] = j ? fmax3(cm[e], x[0], x[1]) : fmaxf(x[0], x[1]);
                    if (NH == 2) cm[e] = fmax3(cm[e], x[2], x[3]);
                }
            }
            if (__any_sync(0xffffffffu, vmx > v_top || cm[0] > thr[0] || cm[1] > thr[1])) {
                // O moves by an exact power of two for the scales, and by what the maxima grew
                const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(vmx));
                float move = 1.f;
                if (__uint_as_float(vb) > v_top) {
                    // (not below 2^-100, where its inverse would leave fp32)
                    const float top = fmaxf(__uint_as_float((vb + 0x7FFFFFu) & 0x7F800000u), kScaleLeast);
                    v_inv = kPUp / top;
                    move = v_top / top;
                    v_top = top;
                }
                float al[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = NH == 1 ? col_max(cm[e]) : quad_max(cm[e]);
                    const float mn = x > thr[e] ? ceilf(x * f0) : mr[e];
                    al[e] = mr[e] == -INFINITY ? 0.f : fast_exp2(mr[e] - mn);
                    mr[e] = mn;
                    thr[e] = (mn + kMaxSlack) / f0;
                    nr[e] = mn == -INFINITY ? 0.f : -mn;
                }
#pragma unroll
                for (int e = 0; e < NH; ++e)
                    ls[e] = fmul2(ls[e], NH == 1 ? make_float2(al[0], al[1]) : make_float2(al[e], al[e]));
                al[0] *= move;
                al[1] *= move;
#pragma unroll
                for (int i = 0; i < 2 * NG * NH; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][e] *= al[NH == 1 ? e & 1 : e >> 1];
            }
            // P, and its products with V, one 16-token k-step per page
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const uint32_t vb = at + j * C::kPageBytes + C::kRec;
                uint32_t vc[NG][2], vz[NG][2];
#pragma unroll
                for (int i = 0; i < NG / 2; ++i) {
                    ldsm_x4_t(vb + 512 * i + 16 * lane, vc[2 * i][0], vc[2 * i][1], vc[2 * i + 1][0], vc[2 * i + 1][1]);
                    ldsm_x4(vb + 8 * D + 64 * i + 16 * (lane >> 3), vz[2 * i][0], vz[2 * i][1], vz[2 * i + 1][0],
                            vz[2 * i + 1][1]);
                }
                const float2 f2 = make_float2(f0, f0), i2 = make_float2(v_inv, v_inv);
                float2 px[2][NH];
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int e = 0; e < NH; ++e) {
                        const float2 x = ffma2(s[j][r][e], f2, NH == 1 ? make_float2(nr[0], nr[1]) : make_float2(nr[e], nr[e]));
                        px[r][e] = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                        ls[e] = fadd2(ls[e], px[r][e]);
                        px[r][e] = fmul2(px[r][e], i2);
                    }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    // codes less z, of the tokens 2 t4, 2 t4 + 1 ([0]) and 8 further ([1]); exact, multiples of 2^-24
                    uint32_t v[4][2];  // even code of byte 0, with 16 odd, the same of byte 1
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        constexpr uint32_t m1 = 0xBC00BC00u, m17 = 0xCC40CC40u;  // -1, -17
                        const uint32_t z = vz[i][r] & kEven, hi = high_bytes(vc[i][r]);
                        v[0][r] = fma_h2(z, m1, vc[i][r] & kEven);
                        v[1][r] = fma_h2(z, m17, vc[i][r] & kBoth);
                        v[2][r] = fma_h2(z, m1, hi & kEven);
                        v[3][r] = fma_h2(z, m17, hi);
                    }
                    if (NH == 1) {
                        // P^T fragments: transpose (token, head) blocks to (head, token)
                        const float s0 = vs[j][i][0].x, s1 = vs[j][i][0].y;
                        const uint32_t b0 = movmatrix_t(pack_f16x2(px[0][0].x * s0, px[0][0].y * s0));
                        const uint32_t b1 = movmatrix_t(pack_f16x2(px[1][0].x * s1, px[1][0].y * s1));
                        mma_f16_16816(acc[2 * i], v[0][0], v[1][0], v[0][1], v[1][1], b0, b1);
                        mma_f16_16816(acc[2 * i + 1], v[2][0], v[3][0], v[2][1], v[3][1], b0, b1);
                    } else {
                        uint32_t p[2][2];  // [token half][head half]
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int e = 0; e < NH; ++e) {
                                const float2 x = fmul2(px[r][e], vs[j][i][r]);
                                p[r][e] = pack_f16x2(x.x, x.y);
                            }
#pragma unroll
                        for (int n = 0; n < 4; ++n)
                            mma_f16_16816(acc[(4 * i + n) % (2 * NG * NH)], p[0][0], p[0][1], p[1][0], p[1][1], v[n][0], v[n][1]);
                    }
                }
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        produce(stage);

        if (cur.z & kEnd) {
            const bool whole = cur.z & kWhole;
            const int64_t slot = (int64_t)wglob + (int64_t)cur.x * a.Hkv + cur.y;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float L = NH == 1 ? col_sum(e ? ls[0].y : ls[0].x) : quad_sum(ls[e * (NH - 1)].x + ls[e * (NH - 1)].y);
                const int hc = NH == 1 ? 2 * t4 + e : gr + 8 * e;  // head in the group
                const int h = cur.y * a.G + hc;
                const float m = mr[e];
                float scl = kStateDown, lse2 = -INFINITY;
                if (whole) {
                    const float sk = a.sinks && hc < a.G ? a.sinks[h] * kLog2e : -INFINITY;
                    const float M = fmaxf(m, sk);
                    scl = 0.f;
                    if (M != -INFINITY) {
                        const float wm = m == -INFINITY ? 0.f : exp2f(m - M);
                        const float den = L * wm + (sk == -INFINITY ? 0.f : exp2f(sk - M));
                        scl = wm / den;
                        lse2 = M + log2f(den);
                    }
                }
                const float up = kUp24 / kPUp * scl;
                // the channels of an m-tile's (8 heads) or two n-tiles' (16) even codes, and odd ones
                auto even = [&](float x) { return x * up * v_top; };
                auto odd = [&](float both, float x) { return (both - x) * 0.0625f * up * v_top; };
                auto put = [&](int ch, float4 v) {  // four channels from ch on
                    if (hc >= a.G) return;
                    if (whole)
                        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + ((int64_t)cur.x * a.Hq + h) * D +
                                                   ch) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                    else
                        *reinterpret_cast<float4 *>(a.part_acc + (slot * a.G + hc) * D + ch) = v;
                };
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    if (NH == 1) {
                        // this lane's channels of the group: 8 (gr / 2) + gr % 2 + 0, 2, 4, 6; the lane beside
                        // it has those between.  The even one takes the first four, the odd one the others.
                        const float c0 = even(acc[2 * i][e]), c2 = odd(acc[2 * i][2 + e], acc[2 * i][e]);
                        const float c4 = even(acc[2 * i + 1][e]), c6 = odd(acc[2 * i + 1][2 + e], acc[2 * i + 1][e]);
                        const bool second = gr & 1;
                        const float r0 = __shfl_xor_sync(0xffffffffu, second ? c0 : c4, 4);
                        const float r1 = __shfl_xor_sync(0xffffffffu, second ? c2 : c6, 4);
                        put(32 * i + 4 * gr, second ? make_float4(r0, c4, r1, c6) : make_float4(c0, r0, c2, r1));
                    } else {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float(&y)[4] = acc[(4 * i + 2 * x) % (2 * NG * NH)], (&b)[4] = acc[(4 * i + 2 * x + 1) % (2 * NG * NH)];
                            put(32 * i + 8 * t4 + 4 * x, make_float4(even(y[2 * e]), even(y[2 * e + 1]), odd(b[2 * e], y[2 * e]),
                                                                     odd(b[2 * e + 1], y[2 * e + 1])));
                        }
                    }
                }
                if (hc >= a.G || (NH == 1 ? gr : t4) != 0) continue;
                if (!whole)
                    *reinterpret_cast<float2 *>(a.part_ml + (slot * a.G + hc) * 2) =
                        make_float2(m + kMaxSlack, L * kStateDown);
                else if (a.lse)
                    a.lse[(int64_t)cur.x * a.Hq + h] = lse2 * kLn2;
            }
        }
    }
    // Near the end of the grid the merge may take its place on the SMs; it waits for this grid before
    // it reads.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int D, int NH>
cudaError_t int4_shape_for(int B, int device, int *ctas, int *warps, int *smem) {
    using C = Int4Cfg<D, NH>;
    const int bytes = int4_smem_bytes<D, NH>(B);
    int optin = 0, sms = 0, occ = 1 << 30;
    cudaError_t e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return e;
    const void *kernels[2] = {reinterpret_cast<const void *>(decode_int4_kernel<D, NH, false>),
                              reinterpret_cast<const void *>(decode_int4_kernel<D, NH, true>)};
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

cudaError_t decode_int4_launch_shape(int D, int G, int B, int device, int *ctas, int *warps_per_cta,
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
        e = int4_shape_for<64, 1>(B, device, ctas, warps_per_cta, smem_bytes);
    else if (D == 64)
        e = int4_shape_for<64, 2>(B, device, ctas, warps_per_cta, smem_bytes);
    else if (D == 128 && NH == 1)
        e = int4_shape_for<128, 1>(B, device, ctas, warps_per_cta, smem_bytes);
    else if (D == 128)
        e = int4_shape_for<128, 2>(B, device, ctas, warps_per_cta, smem_bytes);
    else
        return cudaErrorInvalidValue;
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> lock(mu);
        if (cache.size() > 256) cache.clear();
        cache.push_back({device, D, NH, B, *ctas, *warps_per_cta, *smem_bytes});
    }
    return e;
}

cudaError_t launch_decode_int4(int D, const DecodeArgs &a, int ctas, int smem_bytes, cudaStream_t stream) {
    const bool w = a.window > 0, two = a.G > 8;
#define SINKATTN_INT4_LAUNCH(DD, NN, WW) \
    decode_int4_kernel<DD, NN, WW><<<ctas, Int4Cfg<DD, NN>::kThreads, smem_bytes, stream>>>(a)
    if (D == 64) {
        if (two) {
            if (w) SINKATTN_INT4_LAUNCH(64, 2, true); else SINKATTN_INT4_LAUNCH(64, 2, false);
        } else {
            if (w) SINKATTN_INT4_LAUNCH(64, 1, true); else SINKATTN_INT4_LAUNCH(64, 1, false);
        }
    } else {
        if (two) {
            if (w) SINKATTN_INT4_LAUNCH(128, 2, true); else SINKATTN_INT4_LAUNCH(128, 2, false);
        } else {
            if (w) SINKATTN_INT4_LAUNCH(128, 1, true); else SINKATTN_INT4_LAUNCH(128, 1, false);
        }
    }
#undef SINKATTN_INT4_LAUNCH
    return cudaGetLastError();
}

}  // namespace sinkattn
