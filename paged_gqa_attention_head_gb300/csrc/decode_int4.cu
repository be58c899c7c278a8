// Split-KV paged decode with per-head sinks over a 4-bit cache (append_int4.cu): value = s (code - z)
// with a scale s and a zero code z for every token and 32 channels.
//
// The plan and the products are those of the INT8 decode: every warp takes an equal run of units,
// S^T = K Q^T and O^T = V^T P^T on m16n8k16 f16 MMAs with the 16 tokens of a page, then head_dim, on
// the M axis and the query heads on N, and a merge of the split sequences' states.  A page's K and V
// of a head are one contiguous record of 18 D bytes, copied by one untiled bulk copy.
// What four bits change is the arithmetic that a byte of the cache brings, so that is what the layout
// and the kernel save on:
//   * a code is taken as the f16 subnormal code * 2^-24: a 32-bit word of eight codes becomes four
//     operand registers with four ANDs and one shift.  Every other pair stays four bits up, 16 times
//     its value: for K the query's entries are a sixteenth there, for V the output rows are divided
//     at the end.  The contraction runs over channels in the word's order, which is the query's too;
//   * V comes by transposing 8x8 loads of 16-bit elements, four channels of a token: a register holds
//     the same four channels of two neighbouring tokens, and the ANDs part the channels;
//   * the words of a page come by 8x8 loads whose eight row addresses are the same: transposed,
//     a lane gets its own token's word twice (the scale as a float: one AND; z as an f16 pair:
//     another), plain, the words of its two neighbouring tokens (z as the pair that V needs);
//   * z comes off on the tensor cores: for K a product of z with -sum of the group's q (in two f16
//     parts), which the group's code products start from; for V one product of z with the group's P,
//     subtracted once a step;
//   * a group's K scores are multiplied by s in fp32 pairs; P of a group is taken times s, relative to
//     the power of two above the largest V scale met, and rounded once to f16, as in the INT8 decode.
// The running maximum moves only when a score passes it by more than 8 (log2), as there.
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
    static constexpr int kPPU = D == 64 ? 8 : 4;               // pages of a unit: one copy stage of 9 KB
    static constexpr int kStep = D == 64 && NH == 1 ? 4 : 2;   // pages whose scores are held at once
    static constexpr int kStages = 2;
    static constexpr int kRec = 9 * D;                         // K (or V) of a (page, head)
    static constexpr int kPageBytes = 2 * kRec;
    static constexpr int kStageBytes = kPPU * kPageBytes;
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kGroups = D / 32;
    static constexpr int kCtas = NH == 2 && D == 128 ? 2 : 3;  // CTAs an SM, by registers
};

constexpr float kPShift = 7.f;   // P = 2^(s - m + kPShift)
constexpr float kMaxSlack = 8.f; // the running maximum moves when a score passes it by more
constexpr float kStateDown = 1.f / 32768.f;  // states leave with their sums over 2^(kPShift + kMaxSlack)
constexpr float kUp24 = 16777216.f;          // 2^24
constexpr uint32_t kEven = 0x000F000Fu, kOdd = 0x00F000F0u;  // pairs of codes in place, and 16 times them

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
    return min(max(a.seq_lens[b], 0), a.max_pages * kPageSize);
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

__device__ __forceinline__ float f16_of(float x) {  // rounded to f16
    float y;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.f16.f32 h, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(y) : "f"(x));
    return y;
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

    // The copy side's position, its sequence's length, the first unit of its segment, and the units
    // copied so far.
    Cursor pc;
    {
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
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
    int pL = length_of(a, pc.b), p_seg0 = pc.p, produced = 0;

    // Block-table window: lane l holds the entry of visible page win_p0 + l of sequence win_b (-1 past
    // its last page); the entries of the next 32 pages are loaded with it.
    int win_b = -1, win_p0 = 0, win_val = -1, nxt_val = -1;
    auto entry = [&](int b, int first, int npv, int q) {
        return q < npv ? a.block_table[(int64_t)b * a.max_pages + first + q] : -1;
    };
    const uint64_t policy = l2_policy_evict_first();
    // The next unit, if there is one, into a stage: lanes 0 .. U - 1 take a page each.
    auto produce = [&](int stage) {
        if (produced == n_units) return;
        const Cursor c = pc;
        const int L = pL;
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
                if (pc.b < a.B) pL = length_of(a, pc.b);
            }
        }
        const int first = first_page<kWindow>(a, L);
        const int npv = (L + kPageSize - 1) / kPageSize - first;  // pages the query sees
        const int pp0 = c.p * U, p0 = pp0 & ~31;
        if (c.b != win_b || p0 != win_p0) {  // warp-uniform
            win_val = c.b == win_b && p0 == win_p0 + 32 ? nxt_val : entry(c.b, first, npv, p0 + lane);
            nxt_val = entry(c.b, first, npv, p0 + 32 + lane);
            win_b = c.b;
            win_p0 = p0;
        }
        const int pg = __shfl_sync(0xffffffffu, win_val, (pp0 + (lane & (U - 1))) & 31);
        const bool in = lane < U && pp0 + lane < npv, ok = in && pg >= 0 && pg < a.num_pages;
        if (in && !ok) set_status(a.status, SINKATTN_STATUS_BAD_PAGE);
        const uint32_t oks = __ballot_sync(0xffffffffu, ok);
        uint64_t *bar = &wbar[stage];
        if (lane == 0) {
            const int key0 = kPageSize * (first + pp0);  // position of the unit's first key
            UnitMeta4 &m = wunit[stage];
            *reinterpret_cast<int4 *>(&m.b) = make_int4(c.b, c.g, flags, (int)oks);
            *reinterpret_cast<int2 *>(&m.end) = make_int2(L - key0, kWindow ? L - a.window - key0 : 0);
            if (oks)
                mbar_arrive_expect_tx(bar, __popc(oks) * C::kPageBytes);
            else
                mbar_arrive(bar);
        }
        __syncwarp();
        if (ok)
            bulk_load_hint(wbuf + stage * C::kStageBytes + lane * C::kPageBytes,
                           static_cast<const uint8_t *>(a.kv_int4) + ((int64_t)pg * a.Hkv + c.g) * C::kPageBytes,
                           C::kPageBytes, bar, policy);
    };

#pragma unroll 1
    for (int st = 0; st < S; ++st) produce(st);

    const int gr = lane >> 2, t4 = lane & 3;
    uint32_t qf[2 * NG][NH][2];
    uint32_t qz[NG][NH];              // -sum of the group's q as two f16 parts (lanes t4 = 0, else 0)
    float acc[2 * NG][NH][4];         // O^T * 2^-24: rows 32g + 8 (gr / 2) + gr % 2 + 4x, 16 times those 2 further
    float mr[NH][2];                  // running maximum of the scores (log2)
    float2 nr[NH], ls[NH];            // -(mr - kPShift), 0 before the first key; sums of P
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
            // q times 2^(9 - e), e the exponent of the group's largest entry (kept where both powers are
            // normal floats), with the sign of the score scale: sums of 32 stay in f16
            const int ex = min(max((int)(__reduce_max_sync(0xffffffffu, mx) >> 7), 20), 254);
            const float down = copysignf(__uint_as_float((uint32_t)(263 - ex) << 23), a.scale_log2);
            // (never 0, so that a hidden key's -inf stays one)
            f0 = fmaxf(fabsf(a.scale_log2) * __uint_as_float((uint32_t)(ex - 9) << 23) * kUp24, 1e-37f);
#pragma unroll
            for (int kk = 0; kk < 2 * NG; ++kk)
#pragma unroll
                for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t w = qf[kk][nt][e];
                        const float d = e ? down * 0.0625f : down;
                        qf[kk][nt][e] = pack_f16x2(__uint_as_float(w << 16) * d, __uint_as_float(w & 0xFFFF0000u) * d);
                    }
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int nt = 0; nt < NH; ++nt) {
                    // sum of the group's q as the codes meet it: every row the same, columns 2 t4, 2 t4 + 1
                    constexpr uint32_t one = 0x00010001u, one16 = 0x00100010u;
                    float o[4];
                    mma_f16_16816_from(o, 0.f, 0.f, one, one, one16, one16, qf[2 * i][nt][0], qf[2 * i][nt][1]);
                    mma_f16_16816(o, one, one, one16, one16, qf[2 * i + 1][nt][0], qf[2 * i + 1][nt][1]);
                    const float x = __shfl_sync(0xffffffffu, o[0], gr >> 1), y = __shfl_sync(0xffffffffu, o[1], gr >> 1);
                    const float neg = -((gr & 1) ? y : x) * kUp24, hi = f16_of(neg);
                    qz[i][nt] = t4 == 0 ? pack_f16x2(hi, neg - hi) : 0u;
                }
#pragma unroll
            for (int mt = 0; mt < 2 * NG; ++mt)
#pragma unroll
                for (int nt = 0; nt < NH; ++nt)
                    acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.f;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                mr[nt][0] = mr[nt][1] = -INFINITY;
                nr[nt] = ls[nt] = make_float2(0.f, 0.f);
            }
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

            // S^T = K Q^T per page: rows tokens, columns heads; a group's part times its tokens' scales
            float2 s[W][NH][2];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const uint32_t kb = at + j * C::kPageBytes;
                uint32_t kc[NG][2], kw[NG][2];
#pragma unroll
                for (int i = 0; i < NG / 2; ++i) {
                    ldsm_x4(kb + 512 * i + 16 * lane, kc[2 * i][0], kc[2 * i][1], kc[2 * i + 1][0], kc[2 * i + 1][1]);
                    ldsm_x4_t(kb + 8 * D + 64 * i + 16 * (lane >> 3), kw[2 * i][0], kw[2 * i][1], kw[2 * i + 1][0],
                              kw[2 * i + 1][1]);
                }
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const uint32_t w0 = kc[i][0], w1 = kc[i][1], h0 = w0 >> 8, h1 = w1 >> 8;
                    const float s0 = __uint_as_float(kw[i][0] & 0xFFF00000u), s1 = __uint_as_float(kw[i][1] & 0xFFF00000u);
#pragma unroll
                    for (int nt = 0; nt < NH; ++nt) {
                        float o[4];
                        mma_f16_16816_from(o, 0.f, 0.f, kw[i][0] & kEven, kw[i][1] & kEven, 0u, 0u, qz[i][nt], 0u);
                        mma_f16_16816(o, w0 & kEven, w1 & kEven, w0 & kOdd, w1 & kOdd, qf[2 * i][nt][0], qf[2 * i][nt][1]);
                        mma_f16_16816(o, h0 & kEven, h1 & kEven, h0 & kOdd, h1 & kOdd, qf[2 * i + 1][nt][0],
                                      qf[2 * i + 1][nt][1]);
                        const float2 x = make_float2(o[0], o[1]), y = make_float2(o[2], o[3]);
                        s[j][nt][0] = i ? ffma2(x, make_float2(s0, s0), s[j][nt][0]) : fmul2(x, make_float2(s0, s0));
                        s[j][nt][1] = i ? ffma2(y, make_float2(s1, s1), s[j][nt][1]) : fmul2(y, make_float2(s1, s1));
                    }
                }
                if (ragged) {
                    const int n = nv(j), l = lo(j);
                    const bool ok0 = gr < n && gr >= l, ok1 = gr + 8 < n && gr + 8 >= l;
#pragma unroll
                    for (int nt = 0; nt < NH; ++nt) {
                        if (!ok0) s[j][nt][0] = make_float2(-INFINITY, -INFINITY);
                        if (!ok1) s[j][nt][1] = make_float2(-INFINITY, -INFINITY);
                    }
                }
            }
            // V scales of the lane's tokens
            float vs[W][NG][2];
            float vmx = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                uint32_t w[NG][2];
#pragma unroll
                for (int i = 0; i < NG / 2; ++i)
                    ldsm_x4_t(at + j * C::kPageBytes + C::kRec + 8 * D + 64 * i + 16 * (lane >> 3), w[2 * i][0], w[2 * i][1],
                              w[2 * i + 1][0], w[2 * i + 1][1]);
                const int n = nv(j), l = lo(j);
#pragma unroll
                for (int i = 0; i < NG; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (ragged && (gr + 8 * r >= n || gr + 8 * r < l)) w[i][r] = 0;  // whatever lies there
                        vs[j][i][r] = __uint_as_float(w[i][r] & 0xFFF00000u);
                    }
#pragma unroll
                for (int i = 0; i < NG; ++i) vmx = fmax3(vmx, vs[j][i][0], vs[j][i][1]);
            }
            // a score too far above the running maximum, or a V scale above every one so far
            float cm[NH][2];
            bool raise = vmx > v_top;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt) {
                cm[nt][0] = fmaxf(s[0][nt][0].x, s[0][nt][1].x);
                cm[nt][1] = fmaxf(s[0][nt][0].y, s[0][nt][1].y);
#pragma unroll
                for (int j = 1; j < W; ++j) {
                    cm[nt][0] = fmax3(cm[nt][0], s[j][nt][0].x, s[j][nt][1].x);
                    cm[nt][1] = fmax3(cm[nt][1], s[j][nt][0].y, s[j][nt][1].y);
                }
                raise |= cm[nt][0] * f0 > mr[nt][0] + kMaxSlack || cm[nt][1] * f0 > mr[nt][1] + kMaxSlack;
            }
            if (__any_sync(0xffffffffu, raise)) {
                // O^T moves by an exact power of two for the scales, and by what the maxima grew
                const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(vmx));
                float move = 1.f;
                if (__uint_as_float(vb) > v_top) {
                    const float top = __uint_as_float((vb + 0x7FFFFFu) & 0x7F800000u);
                    v_inv = 1.0f / top;
                    move = v_top * v_inv;
                    v_top = top;
                }
#pragma unroll
                for (int nt = 0; nt < NH; ++nt) {
                    float al[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = col_max(cm[nt][e]) * f0;
                        const float mn = x > mr[nt][e] + kMaxSlack ? x : mr[nt][e];
                        al[e] = mr[nt][e] == -INFINITY ? 0.f : fast_exp2(mr[nt][e] - mn);
                        mr[nt][e] = mn;
                    }
                    nr[nt] = make_float2(mr[nt][0] == -INFINITY ? 0.f : kPShift - mr[nt][0],
                                         mr[nt][1] == -INFINITY ? 0.f : kPShift - mr[nt][1]);
                    ls[nt] = fmul2(ls[nt], make_float2(al[0], al[1]));
                    al[0] *= move;
                    al[1] *= move;
#pragma unroll
                    for (int mt = 0; mt < 2 * NG; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[mt][nt][e] *= al[e & 1];
                }
            }
            // P, and O^T += V^T P^T, one 16-token k-step per page
            float od[NG][NH][4];  // what z takes off, rows all the same
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
#pragma unroll
                for (int nt = 0; nt < NH; ++nt) {
                    const float2 f2 = make_float2(f0, f0), i2 = make_float2(v_inv, v_inv);
                    float2 x = ffma2(s[j][nt][0], f2, nr[nt]), y = ffma2(s[j][nt][1], f2, nr[nt]);
                    x = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    ls[nt] = fadd2(ls[nt], fadd2(x, y));
                    x = fmul2(x, i2);
                    y = fmul2(y, i2);
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        const float2 p = fmul2(x, make_float2(vs[j][i][0], vs[j][i][0]));
                        const float2 q = fmul2(y, make_float2(vs[j][i][1], vs[j][i][1]));
                        // P^T fragments: transpose (token, head) blocks to (head, token)
                        const uint32_t b0 = movmatrix_t(pack_f16x2(p.x, p.y)), b1 = movmatrix_t(pack_f16x2(q.x, q.y));
                        const uint32_t z0 = vz[i][0] & kEven, z1 = vz[i][1] & kEven;
                        if (j == 0)
                            mma_f16_16816_from(od[i][nt], 0.f, 0.f, z0, z0, z1, z1, b0, b1);
                        else
                            mma_f16_16816(od[i][nt], z0, z0, z1, z1, b0, b1);
                        const uint32_t w0 = vc[i][0], w1 = vc[i][1], h0 = w0 >> 8, h1 = w1 >> 8;
                        mma_f16_16816(acc[2 * i][nt], w0 & kEven, w0 & kOdd, w1 & kEven, w1 & kOdd, b0, b1);
                        mma_f16_16816(acc[2 * i + 1][nt], h0 & kEven, h0 & kOdd, h1 & kEven, h1 & kOdd, b0, b1);
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < 2 * NG; ++mt)
#pragma unroll
                for (int nt = 0; nt < NH; ++nt) {
                    const float2 o = make_float2(od[mt / 2][nt][0], od[mt / 2][nt][1]);
                    const float2 x = ffma2(o, make_float2(-1.f, -1.f), make_float2(acc[mt][nt][0], acc[mt][nt][1]));
                    const float2 y = ffma2(o, make_float2(-16.f, -16.f), make_float2(acc[mt][nt][2], acc[mt][nt][3]));
                    acc[mt][nt][0] = x.x;
                    acc[mt][nt][1] = x.y;
                    acc[mt][nt][2] = y.x;
                    acc[mt][nt][3] = y.y;
                }
        }
        fence_proxy_async_smem();
        __syncwarp();
        produce(stage);

        if (cur.z & kEnd) {
            const bool whole = cur.z & kWhole;
            const int64_t slot = (int64_t)wglob + (int64_t)cur.x * a.Hkv + cur.y;
#pragma unroll
            for (int nt = 0; nt < NH; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float L = col_sum(e ? ls[nt].y : ls[nt].x);
                    const int hc = nt * 8 + 2 * t4 + e;  // column (head in the group)
                    const int h = cur.y * a.G + hc;
                    // reference of the state: probabilities were taken against mr - kPShift
                    const float m = mr[nt][e] == -INFINITY ? -INFINITY : mr[nt][e] - kPShift;
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
                    const float up = kUp24 * scl;
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        // this lane's channels of the group: 8 (gr / 2) + gr % 2 + 0, 2, 4, 6; the lane
                        // beside it has those between.  The even one takes the first four, the odd one
                        // the others.
                        const float c0 = acc[2 * i][nt][e] * up * v_top, c2 = acc[2 * i][nt][2 + e] * 0.0625f * up * v_top;
                        const float c4 = acc[2 * i + 1][nt][e] * up * v_top;
                        const float c6 = acc[2 * i + 1][nt][2 + e] * 0.0625f * up * v_top;
                        const bool odd = gr & 1;
                        const float r0 = __shfl_xor_sync(0xffffffffu, odd ? c0 : c4, 4);
                        const float r1 = __shfl_xor_sync(0xffffffffu, odd ? c2 : c6, 4);
                        const float4 v = odd ? make_float4(r0, c4, r1, c6) : make_float4(c0, r0, c2, r1);
                        if (hc >= a.G) continue;
                        const int ch = 32 * i + 4 * gr;
                        if (whole)
                            *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) +
                                                       ((int64_t)cur.x * a.Hq + h) * D + ch) =
                                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4 *>(a.part_acc + (slot * a.G + hc) * D + ch) = v;
                    }
                    if (hc >= a.G || gr != 0) continue;
                    if (!whole)
                        *reinterpret_cast<float2 *>(a.part_ml + (slot * a.G + hc) * 2) =
                            make_float2(m + kPShift + kMaxSlack, L * kStateDown);
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
