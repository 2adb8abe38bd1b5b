// Attention over the paged 8-bit cache for few query rows per key/value head
// (decode steps, a handful of speculated tokens): bound by reading the cache.
//
// For a row with query q, tokens t it may see, e4m3 keys k_t and values v_t and
// their pages' scales K, V (one pair per page and head):
//     o = sum_t exp(s_t) V v_t / sum_t exp(s_t),   s_t = scale K (q . k_t).
// Everything runs in base 2, and V goes into the exponent: with
// w_t = 2^(s_t log2 e + log2 V - m + kShift) the sums are O = sum w_t v_t and
// l = sum w_t / V, one pass with a running m, and o = O / l.  So the bytes of
// the cache meet the tensor cores as they are, converted to half precision
// (exactly), and no scale touches a key or value.
//
// Half precision, not bf16, for w and q: eleven bits instead of eight, and its
// range suffices.  m follows the running maximum only when that grew by more
// than kSlack, so w <= 2^(kShift + kSlack) = 2^15; the least half is 2^-24, so a
// token is lost only under 2^-35 of the largest, and l, in fp32, has it still.
// A query row is divided by a power of two first, so that its largest element is
// near 1.
//
// The rows of a (sequence, key/value head), at most 16 at a time (one
// mma.m16n8k16 tile; a decode step has h_q / h_kv of them), are a unit of
// ceil(tokens / 64) blocks.  All units' blocks form one line, and CTA c takes
// its c-th equal part, so unequal lengths are balanced to a block.  A unit that
// lies in several parts is joined by whichever CTA finishes last, from partial
// sums in the workspace, in the order of the parts: the bits do not depend on
// who that is.
//
// A CTA: one warp that issues TMA loads of whole pages into a ring of 64-token
// stages (128-byte swizzle, which makes every fragment load below free of bank
// conflicts), and eight warps that each take 16 tokens of every other stage
// with softmax state of their own; they are joined once per unit.
#include "paged_attention.cuh"

namespace sr {
namespace paged {
namespace {

constexpr int kWarps = 8;              // consumer warps; a warpgroup beside them loads
constexpr int kThreads = 32 * (kWarps + 4);
// Registers of the split: 128 x 40 + 256 x 232 = 384 x 168, what the block is launched with.
constexpr int kLaunchRegs = 168, kLoadRegs = 40, kMathRegs = 232;
static_assert(128 * kLoadRegs + 32 * kWarps * kMathRegs <= kThreads * kLaunchRegs, "the split draws on the launch's registers");
constexpr int kTok = 64;               // tokens per stage: 4 warps of 16
constexpr int kMinBlocks = 2;          // least blocks worth a CTA of their own
constexpr int kUnitStart = 256;         // what a unit costs beside its blocks, in tokens

// Join barrier of the eight consumer warps.
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;\n" ::: "memory"); }
__device__ __forceinline__ bool consumers_or(bool x) {
    int r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.s32 p, %1, 0;\nbar.red.or.pred q, 1, 256, p;\nselp.s32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(int(x))
        : "memory");
    return r != 0;
}

// D += A(16x16) B(16x8), half in, fp32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(r.x), "=r"(r.y) : "r"(addr));
    return r;
}

// Where 16-byte chunk `c` of row `r` lies in a stage's tile (TMA swizzles of
// 128-byte and 64-byte rows); a 256-byte row is two tiles of 128 columns.
template <int D> __device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if (D == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return (c >> 3) * (kTok * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Neighbours 4 apart: 0 4 1 5 2 6 3 7.
__device__ __forceinline__ int spread(int n) { return (n >> 1) | ((n & 1) << 2); }
// Column of O that a lane's accumulator of n-tile t stands for, at column n of the tile.
template <int D> __device__ __forceinline__ int column_of(int n, int t) {
    return D == 64 ? 8 * n + t : (t >> 4) * 128 + 16 * spread(n) + (t & 15);
}

template <int D> struct RowsSmem {
    static constexpr int kTile = kTok * D;                  // bytes of a stage's keys, or values
    static constexpr int kStages = 1024 / D;                // 128 KB in flight
    static constexpr int kRegion = 16 * D * 4;              // one warp's O in fp32
    static constexpr int off_join = kStages * 2 * kTile;    // 4 regions
    // the weights of a join of the most parts use the same space
    static constexpr int kJoin = 4 * kRegion > kRowsMaxCtas * 64 ? 4 * kRegion : kRowsMaxCtas * 64;
    static constexpr int off_q = off_join + kJoin;          // query fragments
    static constexpr int off_misc = off_q + 16 * D * 2;
    struct Misc {
        uint64_t full[kStages], empty[kStages];
        float ml[2][kWarps][16];   // running max and sum of each warp's rows
        float row_scale[16];       // factor of q . k of each row
        int row_seen[16];          // tokens each row may see
        float sums[16];
        LinePlace place;
        int ticket;
    };
    static constexpr int bytes = off_misc + int(sizeof(Misc)) + 1024;  // + alignment of the stages
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const __grid_constant__ AttnParams p) {
    using S = RowsSmem<D>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (tc::smem_u32(raw) & 1023)) & 1023);
    typename S::Misc &misc = *reinterpret_cast<typename S::Misc *>(smem + S::off_misc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&misc.full[i], 1);
            tc::mbar_init(&misc.empty[i], 4);
        }
        tc::fence_mbar_init();
    }
    Line<16, kTok, kUnitStart> line;
    if (!line.start<kThreads>(p, (long long)kMinBlocks * kTok * p.group, misc.place)) return;

    const uint32_t stage0 = tc::smem_u32(smem);
    Segment seg;
    int it = 0;  // stages so far

    if (warp >= kWarps) {  // ---- loads
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kLoadRegs));
        if (warp > kWarps) return;
        while (line.next(seg)) {
            for (int b = seg.b0; b < seg.b1; ++b, ++it) {
                const int slot = it % kStages;
                // a page is loaded whole, also where the sequence ends inside it; pages behind its end are not
                const int tok = b * kTok, pieces = p.page < kTok ? min(kTok, seg.kv - tok + p.page - 1) / p.page : 1;
                const int rows = min(p.page, kTok);
                bool ok = true;
                if (lane == 0) {
                    ok = it < kStages || wait_for(&misc.empty[slot], ((it / kStages) - 1) & 1);
                    if (ok)
                        tc::mbar_arrive_expect_tx(&misc.full[slot], pieces * rows * D * 2);
                    else
                        atomicOr(p.status, SR_DEV_TIMEOUT);
                }
                if (!__shfl_sync(0xffffffffu, int(ok), 0)) return;
                if (lane < pieces) {
                    const int at = tok + lane * rows;
                    int page = p.table[(long long)seg.seq * p.max_pages + at / p.page];
                    page = page < 0 || page >= p.n_pages ? 0 : page;  // the sequence's output is not written
                    const int y = (page * p.h_kv + seg.head) * p.page + at % p.page;
                    uint8_t *k = smem + slot * 2 * S::kTile + lane * rows * (D < 128 ? D : 128);
#pragma unroll
                    for (int x = 0; x < D; x += 128) {
                        tc::tma_load_2d(k + x * kTok, &kmap, &misc.full[slot], x, y);
                        tc::tma_load_2d(k + S::kTile + x * kTok, &vmap, &misc.full[slot], x, y);
                    }
                }
            }
        }
        return;
    }

    // ---- softmax and products
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kMathRegs));
    const int r = lane >> 2, j = lane & 3;
    // Token of score column n of a 16-token step, in its half: 128-byte rows are free of bank conflicts where the two
    // rows of a load phase differ by 4, 64-byte rows where they are neighbours.
    auto token_of = [](int n) { return D == 64 ? n : spread(n); };
    int checked = -1;
    bool bad_pages = false;
    bool alive = true;
    while (line.next(seg)) {
        consumers_sync();  // the queries and the join area are free again
        if (checked != seg.seq) {
            bool bad = false;
            const int pages = (seg.kv + p.page - 1) / p.page;
            for (int i = threadIdx.x; i < pages; i += 32 * kWarps) {
                const int page = p.table[(long long)seg.seq * p.max_pages + i];
                bad |= page < 0 || page >= p.n_pages;
            }
            bad_pages = consumers_or(bad);
            if (bad_pages && threadIdx.x == 0) atomicOr(p.status, SR_DEV_BAD_INDEX);
            checked = seg.seq;
        }
        // query rows 2 warp, 2 warp + 1, divided by a power of two, in fragment order
        uint32_t *qf = reinterpret_cast<uint32_t *>(smem + S::off_q);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = 2 * warp + i;
            constexpr int kPairs = D / 64;  // element pairs per lane
            float2 f[kPairs];
            float top = 0.f;
            const int g = seg.tile * 16 + row, token = g / p.group;
            const __nv_bfloat16 *src = p.q + (long long)(seg.bos + token) * p.q_stride + (seg.head * p.group + g % p.group) * D;
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                f[k] = row < seg.rows ? __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(src)[lane + 32 * k])
                                      : make_float2(0.f, 0.f);
                top = fmaxf(top, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float down = row_down(top);
#pragma unroll
            for (int k = 0; k < kPairs; ++k) {
                const __half2 h = __floats2half2_rn(f[k].x * down, f[k].y * down);
                const int e = 2 * (lane + 32 * k);
                const int step = (e >> 6) * 4 + ((e >> 2) & 3), reg = ((e >> 1) & 1) * 2 + (row >> 3);
                qf[(step * 32 + (row & 7) * 4 + ((e >> 4) & 3)) * 4 + reg] = *reinterpret_cast<const uint32_t *>(&h);
            }
            if (lane == 0) {
                misc.row_scale[row] = p.scale_log2 / down;
                misc.row_seen[row] = row < seg.rows ? max(0, seg.kv - seg.count + token + 1) : 0;
            }
        }
        consumers_sync();

        const float c0 = misc.row_scale[r], c1 = misc.row_scale[r + 8];
        const int seen0 = misc.row_seen[r], seen1 = misc.row_seen[r + 8];
        const int seen_most = misc.row_seen[seg.rows - 1], seen_least = misc.row_seen[0];
        float O[D / 8][4];
#pragma unroll
        for (int t = 0; t < D / 8; ++t) O[t][0] = O[t][1] = O[t][2] = O[t][3] = 0.f;
        float m0 = kNone, m1 = kNone, l0 = 0.f, l1 = 0.f;

        for (int b = seg.b0; b < seg.b1; ++b, ++it) {
            if ((it & 1) != (warp >> 2)) continue;
            const int slot = it % kStages;
            const int row0 = (warp & 3) * 16, tok0 = b * kTok + row0;
            if (alive && !wait_for(&misc.full[slot], (it / kStages) & 1)) {
                if (lane == 0) atomicOr(p.status, SR_DEV_TIMEOUT);
                alive = false;
            }
            if (tok0 < seen_most && alive) {
                const uint32_t kt = stage0 + slot * 2 * S::kTile, vt = kt + S::kTile;
                int page = p.table[(long long)seg.seq * p.max_pages + (tok0 >> p.page_shift)];
                page = page < 0 || page >= p.n_pages ? 0 : page;
                const long long block = (long long)page * p.h_kv + seg.head;
                const float ks = usable_scale(p.k_scale[block]), vs = usable_scale(p.v_scale[block]);

                float s[2][4] = {};
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int row = row0 + 8 * n + token_of(r);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 w = lds128(kt + chunk_at<D>(row, 4 * c + j));
                        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 a = *reinterpret_cast<const uint4 *>(qf + ((c * 4 + i) * 32 + lane) * 4);
                            uint32_t b0, b1;
                            e4m3x4_to_f16x4(words[i], b0, b1);
                            mma_f16(s[n], a, b0, b1);
                        }
                    }
                }
                // values of the tokens of this lane's score columns: two per half
                constexpr int kWords = D / 32;  // words of a token row per lane
                uint32_t v[4][kWords];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = row0 + 8 * (i >> 1) + token_of(2 * j + (i & 1));
                    if (D == 64) {
                        const uint2 w = lds64(vt + chunk_at<D>(row, r >> 1) + (r & 1) * 8);
                        v[i][0] = w.x, v[i][1] = w.y;
                    } else {
#pragma unroll
                        for (int x = 0; x < D / 128; ++x) {
                            const uint4 w = lds128(vt + chunk_at<D>(row, x * 8 + spread(r)));
                            v[i][4 * x] = w.x, v[i][4 * x + 1] = w.y, v[i][4 * x + 2] = w.z, v[i][4 * x + 3] = w.w;
                        }
                    }
                }
                const bool edge = tok0 + 16 > seen_least;
                const float lvs = __log2f(vs), k0 = c0 * ks, k1 = c1 * ks;
                float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = tok0 + 8 * n + token_of(2 * j + e);
                        s[n][e] = fmaf(s[n][e], k0, lvs);
                        s[n][2 + e] = fmaf(s[n][2 + e], k1, lvs);
                        if (edge) {
                            if (t >= seen0) s[n][e] = -INFINITY;
                            if (t >= seen1) s[n][2 + e] = -INFINITY;
                            if (t >= seen_most)  // 0 times a NaN that nobody sees
#pragma unroll
                                for (int w = 0; w < kWords; ++w) v[2 * n + e][w] = 0;
                        }
                        top0 = fmaxf(top0, s[n][e]);
                        top1 = fmaxf(top1, s[n][2 + e]);
                    }
                bool poison = false;
                if (edge && seen_least < seen_most) {  // a NaN that some rows see and others do not
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int w = 0; w < kWords; ++w)
                            if (has_nan(v[i][w])) poison = true, v[i][w] = without_nan(v[i][w]);
                    poison = __any_sync(0xffffffffu, poison);
                }
                top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 1));
                top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
                top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 2));
                top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 2));
                if (__any_sync(0xffffffffu, top0 > m0 + kSlack || top1 > m1 + kSlack)) {
                    const float n0 = fmaxf(m0, top0), n1 = fmaxf(m1, top1);
                    const float f0 = exp2f(m0 - n0), f1 = exp2f(m1 - n1);
                    m0 = n0, m1 = n1, l0 *= f0, l1 *= f1;
#pragma unroll
                    for (int t = 0; t < D / 8; ++t) O[t][0] *= f0, O[t][1] *= f0, O[t][2] *= f1, O[t][3] *= f1;
                }
                const float z0 = m0 - kShift, z1 = m1 - kShift;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        s[n][e] = ex2(s[n][e] - z0);
                        s[n][2 + e] = ex2(s[n][2 + e] - z1);
                    }
                const float up = __frcp_rn(vs);
                l0 = fmaf((s[0][0] + s[0][1]) + (s[1][0] + s[1][1]), up, l0);
                l1 = fmaf((s[0][2] + s[0][3]) + (s[1][2] + s[1][3]), up, l1);
                const uint4 a = make_uint4(pack_f16(s[0][0], s[0][1]), pack_f16(s[0][2], s[0][3]),
                                           pack_f16(s[1][0], s[1][1]), pack_f16(s[1][2], s[1][3]));
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140), x1 = __byte_perm(v[0][w], v[1][w], 0x7362);
                    const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140), y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
                    uint32_t b[8];
                    e4m3x4_to_f16x4(x0, b[0], b[2]);
                    e4m3x4_to_f16x4(y0, b[1], b[3]);
                    e4m3x4_to_f16x4(x1, b[4], b[6]);
                    e4m3x4_to_f16x4(y1, b[5], b[7]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_f16(O[4 * w + i], a, b[2 * i], b[2 * i + 1]);
                }
                if (poison) {
                    for (int t = 0; t < 16 && tok0 + t < seen_most; ++t) {
                        const bool in0 = tok0 + t < seen0, in1 = tok0 + t < seen1;
#pragma unroll
                        for (int u = 0; u < D / 8; ++u)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int col = column_of<D>(2 * j + e, u);
                                const uint8_t x = smem[slot * 2 * S::kTile + S::kTile + chunk_at<D>(row0 + t, col >> 4) +
                                                       (col & 15)];
                                if ((x & 127) == 127) {
                                    if (in0) O[u][e] = NAN;
                                    if (in1) O[u][2 + e] = NAN;
                                }
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&misc.empty[slot]);
        }

        // ---- join the eight warps: rows' largest m, then sums by halving in a fixed order
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (j == 0) {
            misc.ml[0][warp][r] = m0, misc.ml[0][warp][r + 8] = m1;
            misc.ml[1][warp][r] = l0, misc.ml[1][warp][r + 8] = l1;
        }
        consumers_sync();
        float M0 = kNone, M1 = kNone, L0 = 0.f, L1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M0 = fmaxf(M0, misc.ml[0][w][r]), M1 = fmaxf(M1, misc.ml[0][w][r + 8]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            L0 = fmaf(misc.ml[1][w][r], exp2f(misc.ml[0][w][r] - M0), L0);
            L1 = fmaf(misc.ml[1][w][r + 8], exp2f(misc.ml[0][w][r + 8] - M1), L1);
        }
        const float f0 = exp2f(m0 - M0), f1 = exp2f(m1 - M1);
#pragma unroll
        for (int t = 0; t < D / 8; ++t) O[t][0] *= f0, O[t][1] *= f0, O[t][2] *= f1, O[t][3] *= f1;
        float4 *join = reinterpret_cast<float4 *>(smem + S::off_join);
#pragma unroll
        for (int half = kWarps / 2; half; half >>= 1) {
            if (warp >= half && warp < 2 * half)
#pragma unroll
                for (int t = 0; t < D / 8; ++t)
                    join[((warp - half) * (D / 8) + t) * 32 + lane] = make_float4(O[t][0], O[t][1], O[t][2], O[t][3]);
            consumers_sync();
            if (warp < half)
#pragma unroll
                for (int t = 0; t < D / 8; ++t) {
                    const float4 x = join[(warp * (D / 8) + t) * 32 + lane];
                    O[t][0] += x.x, O[t][1] += x.y, O[t][2] += x.z, O[t][3] += x.w;
                }
            consumers_sync();
        }

        if (warp == 0 && seg.whole && !bad_pages) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = r + 8 * i;
                if (row >= seg.rows) continue;
                const float L = i ? L1 : L0, M = i ? M1 : M0, inv = L == 0.f ? 0.f : 1.f / L;
                const int g = seg.tile * 16 + row;
                const long long at = (long long)(seg.bos + g / p.group) * p.h_q + seg.head * p.group + g % p.group;
                __nv_bfloat16 *out = p.o + at * D;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int t = 0; t < D / 8; t += 4) {
                        const uint32_t lo = pack_bf16(O[t][2 * i + e] * inv, O[t + 1][2 * i + e] * inv);
                        const uint32_t hi = pack_bf16(O[t + 2][2 * i + e] * inv, O[t + 3][2 * i + e] * inv);
                        *reinterpret_cast<uint2 *>(out + column_of<D>(2 * j + e, t)) = make_uint2(lo, hi);
                    }
                if (p.lse && j == 0) p.lse[at] = log_sum(M, L);
            }
        }
        if (!seg.whole) {
            // ---- a part of a unit: to the workspace; the last CTA to come joins all parts
            const int first_cta = line.first_cta(seg), last_cta = line.last_cta(seg);
            const int part_slot = 2 * blockIdx.x + (int(blockIdx.x) == first_cta ? 1 : 0);
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = r + 8 * i;
                    if (row >= seg.rows) continue;
                    float *out = p.parts + ((long long)part_slot * 16 + row) * D;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int t = 0; t < D / 8; t += 4)
                            *reinterpret_cast<float4 *>(out + column_of<D>(2 * j + e, t)) =
                                make_float4(O[t][2 * i + e], O[t + 1][2 * i + e], O[t + 2][2 * i + e], O[t + 3][2 * i + e]);
                    if (j == 0) p.part_ml[part_slot * 16 + row] = make_float2(i ? M1 : M0, i ? L1 : L0);
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const int last = last_cta - first_cta;
                    const bool mine = atomicAdd(&p.tickets[first_cta], 1) == last;
                    if (mine) p.tickets[first_cta] = 0;
                    __threadfence();
                    misc.ticket = mine;
                }
            }
            consumers_sync();
            if (misc.ticket && !bad_pages) {
                const int parts = last_cta - first_cta + 1;
                auto slot_of = [&](int i) { return 2 * (first_cta + i) + (i == 0); };
                float *weight = reinterpret_cast<float *>(smem + S::off_join);  // [16][parts]
                for (int row = warp; row < seg.rows; row += kWarps) {
                    float M = kNone;
                    for (int i = lane; i < parts; i += 32) M = fmaxf(M, __ldcg(&p.part_ml[slot_of(i) * 16 + row]).x);
#pragma unroll
                    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                    float L = 0.f;
                    for (int i = lane; i < parts; i += 32) {
                        const float2 ml = __ldcg(&p.part_ml[slot_of(i) * 16 + row]);
                        const float w = exp2f(ml.x - M);
                        weight[row * parts + i] = w;
                        L = fmaf(ml.y, w, L);
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
                    if (lane == 0) {
                        misc.sums[row] = L == 0.f ? 0.f : 1.f / L;
                        const int g = seg.tile * 16 + row;
                        if (p.lse)
                            p.lse[(long long)(seg.bos + g / p.group) * p.h_q + seg.head * p.group + g % p.group] = log_sum(M, L);
                    }
                }
                consumers_sync();
                for (int i = threadIdx.x; i < seg.rows * (D / 4); i += 32 * kWarps) {
                    const int row = i / (D / 4), c4 = i - row * (D / 4);
                    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (int k = 0; k < parts; ++k) {
                        const float w = weight[row * parts + k];
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(p.parts + ((long long)slot_of(k) * 16 + row) * D) + c4);
                        sum.x = fmaf(w, x.x, sum.x), sum.y = fmaf(w, x.y, sum.y);
                        sum.z = fmaf(w, x.z, sum.z), sum.w = fmaf(w, x.w, sum.w);
                    }
                    const float inv = misc.sums[row];
                    const int g = seg.tile * 16 + row;
                    const long long at = (long long)(seg.bos + g / p.group) * p.h_q + seg.head * p.group + g % p.group;
                    *reinterpret_cast<uint2 *>(p.o + at * D + 4 * c4) =
                        make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
                }
            }
        }
    }
}

template <int D> cudaError_t launch(const CUtensorMap &k, const CUtensorMap &v, AttnParams p, cudaStream_t st) {
    const int bytes = RowsSmem<D>::bytes;
    cudaError_t e = cudaFuncSetAttribute(rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    rows_kernel<D><<<kRowsMaxCtas, kThreads, bytes, st>>>(k, v, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t attend_rows(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int d, cudaStream_t st) {
    return d == 64 ? launch<64>(k, v, p, st) : d == 128 ? launch<128>(k, v, p, st) : launch<256>(k, v, p, st);
}

}  // namespace paged
}  // namespace sr
