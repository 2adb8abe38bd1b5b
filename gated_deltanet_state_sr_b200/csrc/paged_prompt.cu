// Attention over the paged 8-bit cache for many query rows (prompts, the
// unmatched tokens behind a cached prefix): bound by the tensor cores.
//
// The sums, base 2 and the value scale in the exponent, are those of
// paged_rows.cu; here tcgen05 forms them on tiles of 128 rows (row = token *
// group + head of the group) by 128 cached tokens:
//   S = Q K^T   keys stay the e4m3 bytes that TMA brought.  A bf16 query has
//               eight significant bits, two e4m3 numbers have four each: after a
//               division by a power of two that brings the row's largest into
//               128..256, q = hi + lo exactly down to 2^-9 of the largest, and
//               within 2^-17 of the largest below.  Two passes of kind::f8f6f4
//               cost what one of kind::f16 does, and no key is converted.
//   O += P V    weights in half precision in tensor memory (over the scores they
//               came from), values converted to half precision, exactly, into
//               shared memory.  e4m3 weights would do for neither accuracy nor
//               range: many small weights beside a large one add up.
// A CTA walks its part of the line of blocks (paged_attention.cuh).  Its warps:
//   two groups of four: softmax, a row per thread, for two tiles of query rows
//     (head dimension 256: one tile, whose scores have two buffers; its second
//     group is idle), and the queries' split at the start of a unit;
//   one group of four: values to half precision;
//   a warp that issues the products, S of two items ahead of P V of one;
//   a warp that loads pages.
// Tensor memory: two buffers of scores (128 columns each) and the sums O (two
// times 128 columns, or 256).
#include "paged_attention.cuh"

namespace sr {
namespace paged {
namespace {

constexpr int kThreads = 512;
constexpr int kTok = 128;       // cached tokens per tile
constexpr int kHalf = 64;       // tokens per stage of values
constexpr int kMinBlocks = 2;   // least tiles worth a CTA of their own
// 256 x 184 + 128 x 96 + 128 x 48 = 512 x 128, what the block is launched with.
constexpr int kSoftmaxRegs = 184, kConvertRegs = 96, kIssueRegs = 48;
static_assert(256 * kSoftmaxRegs + 128 * kConvertRegs + 128 * kIssueRegs <= 512 * 128, "the split draws on the launch's");
constexpr int kPoisonSlots = 16;

template <int D> struct PromptSmem {
    static constexpr int kTiles = D == 256 ? 1 : 2;            // query tiles
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kSub = D == 64 ? 64 : 128;            // bytes of an 8-bit row in shared memory
    static constexpr int kSubs = D == 256 ? 2 : 1;
    static constexpr int kQ = 128 * D;                         // one part of one query tile
    static constexpr int kK = kTok * D, kKStages = D == 256 ? 2 : 3;
    static constexpr int kRaw = kHalf * D, kRawStages = D == 256 ? 2 : 4;
    static constexpr int kV = kHalf * D * 2, kVStages = D == 256 ? 2 : 4;
    static constexpr int off_k = kTiles * 2 * kQ;
    static constexpr int off_raw = off_k + kKStages * kK;
    static constexpr int off_v = off_raw + kRawStages * kRaw;
    static constexpr int off_misc = off_v + kVStages * kV;
    struct Misc {
        uint64_t q_full, o_free;
        uint64_t k_full[kKStages], k_empty[kKStages];
        uint64_t raw_full[kRawStages], raw_empty[kRawStages];
        uint64_t v_full[kVStages], v_empty[kVStages];
        uint64_t s_full[2], p_full[2], pv_done[2];
        LinePlace place;
        uint32_t tmem;
        int poison[kPoisonSlots];
        int ticket[2];
    };
    static constexpr int bytes = off_misc + int(sizeof(Misc)) + 1024;
};

__device__ __forceinline__ uint64_t sdesc_k_sw64(uint32_t addr) {
    uint64_t d = 0;
    d |= uint64_t((addr >> 4) & 0x3FFF);
    d |= uint64_t(1) << 16;
    d |= uint64_t(512 >> 4) << 32;  // eight rows of 64 bytes
    d |= uint64_t(1) << 46;
    d |= uint64_t(4) << 61;         // 64-byte swizzle
    return d;
}
template <int D> __device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
    return D == 64 ? sdesc_k_sw64(addr) : tc::sdesc_k_sw128(addr);
}
// 16-byte chunk c of row r of an 8-bit tile of `rows` rows.
template <int D> __device__ __forceinline__ uint32_t chunk8_at(int rows, int r, int c) {
    if (D == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Instruction descriptors (D fp32): e4m3 x e4m3, both K-major; half x half, B MN-major.
constexpr uint32_t kIdescS = (1u << 4) | (uint32_t(kTok >> 3) << 17) | (uint32_t(128 >> 4) << 24);
template <int D> constexpr uint32_t idesc_pv() {
    return (1u << 4) | (1u << 16) | (uint32_t(D >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

template <int GROUP> __device__ __forceinline__ void group_sync() {
    asm volatile("bar.sync %0, 128;\n" ::"n"(GROUP) : "memory");
}
__device__ __forceinline__ void softmax_sync(int group) {
    if (group) group_sync<2>(); else group_sync<1>();
}
__device__ __forceinline__ bool softmax_or(int group, bool x) {
    int r;
    if (group)
        asm volatile("{\n.reg .pred p, q;\nsetp.ne.s32 p, %1, 0;\nbar.red.or.pred q, 2, 128, p;\nselp.s32 %0, 1, 0, q;\n}\n"
                     : "=r"(r) : "r"(int(x)) : "memory");
    else
        asm volatile("{\n.reg .pred p, q;\nsetp.ne.s32 p, %1, 0;\nbar.red.or.pred q, 1, 128, p;\nselp.s32 %0, 1, 0, q;\n}\n"
                     : "=r"(r) : "r"(int(x)) : "memory");
    return r != 0;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
    return r;
}

__device__ __forceinline__ int page_at(const AttnParams &p, int seq, int token) {
    const int page = p.table[(long long)seq * p.max_pages + token / p.page];
    return page < 0 || page >= p.n_pages ? 0 : page;  // the output of such a sequence is not written
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ AttnParams p) {
    using S = PromptSmem<D>;
    constexpr int NQ = S::kTiles;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *smem = raw_smem + ((1024 - (tc::smem_u32(raw_smem) & 1023)) & 1023);
    typename S::Misc &misc = *reinterpret_cast<typename S::Misc *>(smem + S::off_misc);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = tc::smem_u32(smem);

    if (threadIdx.x == 0) {
        tc::mbar_init(&misc.q_full, 128 * NQ);
        tc::mbar_init(&misc.o_free, 128 * NQ);
        for (int i = 0; i < S::kKStages; ++i) tc::mbar_init(&misc.k_full[i], 1), tc::mbar_init(&misc.k_empty[i], 1);
        for (int i = 0; i < S::kRawStages; ++i) tc::mbar_init(&misc.raw_full[i], 1), tc::mbar_init(&misc.raw_empty[i], 128);
        for (int i = 0; i < S::kVStages; ++i) tc::mbar_init(&misc.v_full[i], 128), tc::mbar_init(&misc.v_empty[i], 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(&misc.s_full[i], 1), tc::mbar_init(&misc.p_full[i], 128), tc::mbar_init(&misc.pv_done[i], 1);
        for (int i = 0; i < kPoisonSlots; ++i) misc.poison[i] = 0;
        tc::fence_mbar_init();
    }
    Line<S::kRows, kTok> line;
    if (!line.template start<kThreads>(p, kMinBlocks, misc.place)) return;
    if (warp == 12) {
        tc::tmem_alloc(&misc.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = misc.tmem;
    Segment seg;
    bool alive = true;  // a wait that ran out ends a role; the others' waits then run out too
    auto wait = [&](uint64_t &bar, int phase) {
        if (alive && !tc::mbar_wait(&bar, phase & 1)) {
            atomicOr(p.status, SR_DEV_TIMEOUT);
            alive = false;
        }
        return alive;
    };

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kIssueRegs));
        if (warp == 12 && lane == 0) {
            // ---- products
            int kt = 0, vt = 0, w = 0;  // tiles of keys, stages of values, items (tile, query tile) so far
            for (int unit = 0; alive && line.next(seg); ++unit) {
                const int tiles = seg.b1 - seg.b0;
                if (!wait(misc.q_full, unit)) break;
                const int items = tiles * NQ;
                auto scores = [&](int i) {  // item i of the unit: buffer (w + i) & 1
                    const int tile = i / NQ, j = i - tile * NQ, st = (kt + tile) % S::kKStages;
                    if (!wait(misc.k_full[st], (kt + tile) / S::kKStages)) return false;
                    tc::tc_fence_after();
                    const uint32_t d = tmem + ((w + i) & 1) * 128;
                    uint32_t on = 0;
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int s = 0; s < D / 32; ++s) {
                            const uint32_t at = (s * 32 / S::kSub) * 128 * S::kSub + (s * 32) % S::kSub;
                            tc::mma_f8_ss(d, desc_k<D>(base + (j * 2 + part) * S::kQ + at),
                                          desc_k<D>(base + S::off_k + st * S::kK + at), kIdescS, on);
                            on = 1;
                        }
                    tc::mma_commit(&misc.s_full[(w + i) & 1]);
                    if (j == NQ - 1) tc::mma_commit(&misc.k_empty[st]);
                    return true;
                };
                for (int i = 0; i < 2 && i < items; ++i)
                    if (!scores(i)) break;
                if (unit && !wait(misc.o_free, unit - 1)) break;
                for (int i = 0; alive && i < items; ++i) {
                    const int tile = i / NQ, j = i - tile * NQ, b = (w + i) & 1;
                    if (!wait(misc.p_full[b], (w + i) >> 1)) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int n = vt + tile * 2 + h, st = n % S::kVStages;
                        if (!wait(misc.v_full[st], n / S::kVStages)) break;
                        tc::tc_fence_after();
#pragma unroll
                        for (int s = 0; s < kHalf / 16; ++s)
                            mma_f16_ts(tmem + 256 + j * 128, tmem + b * 128 + h * 32 + s * 8,
                                       tc::sdesc_sw128(base + S::off_v + st * S::kV + s * 2048, kHalf * 128, 1024),
                                       idesc_pv<D>(), tile | h | s ? 1u : 0u);
                        if (j == NQ - 1) tc::mma_commit(&misc.v_empty[st]);
                    }
                    if (!alive) break;
                    tc::mma_commit(&misc.pv_done[b]);
                    if (i + 2 < items && !scores(i + 2)) break;
                }
                kt += tiles, vt += 2 * tiles, w += items;
            }
        } else if (warp == 13) {
            // ---- loads: a page (64 rows of it at most) per lane
            int kt = 0, vt = 0;
            const int rows = min(p.page, 64);
            while (line.next(seg)) {
                for (int b = seg.b0; b < seg.b1; ++b, ++kt) {
                    const int ks = kt % S::kKStages;
                    const int left = seg.kv - b * kTok;                      // tokens from here on
                    const int pieces = (min(kTok, left) + rows - 1) / rows;  // pages behind the end are not read
                    const int at = b * kTok + lane * rows;
                    int y = 0;
                    if (lane < pieces) y = (page_at(p, seg.seq, at) * p.h_kv + seg.head) * p.page + at % p.page;
                    int ok = 1;
                    if (lane == 0) {
                        ok = kt < S::kKStages || wait(misc.k_empty[ks], kt / S::kKStages - 1);
                        if (ok) tc::mbar_arrive_expect_tx(&misc.k_full[ks], pieces * rows * D);
                    }
                    if (!__shfl_sync(0xffffffffu, ok, 0)) goto done;
                    if (lane < pieces)
#pragma unroll
                        for (int x = 0; x < S::kSubs; ++x)
                            tc::tma_load_2d(smem + S::off_k + ks * S::kK + x * kTok * 128 + lane * rows * S::kSub, &kmap,
                                            &misc.k_full[ks], x * 128, y);
                    const int per = kHalf / rows;  // pieces per stage of values
#pragma unroll
                    for (int h = 0; h < 2; ++h, ++vt) {
                        const int vs = vt % S::kRawStages;
                        const int mine = min(max(pieces - h * per, 0), per);
                        if (lane == 0) {
                            ok = vt < S::kRawStages || wait(misc.raw_empty[vs], vt / S::kRawStages - 1);
                            if (ok) tc::mbar_arrive_expect_tx(&misc.raw_full[vs], mine * rows * D);
                        }
                        if (!__shfl_sync(0xffffffffu, ok, 0)) goto done;
                        const int l = lane - h * per;
                        if (l >= 0 && l < mine)
#pragma unroll
                            for (int x = 0; x < S::kSubs; ++x)
                                tc::tma_load_2d(smem + S::off_raw + vs * S::kRaw + x * kHalf * 128 + l * rows * S::kSub,
                                                &vmap, &misc.raw_full[vs], x * 128, y);
                    }
                }
            }
        }
    } else if (warp >= 8) {
        // ---- values to half precision: token rows of 64 columns, 128-byte swizzle, the layout of an MN-major operand
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kConvertRegs));
        const int t = threadIdx.x - 256;
        int vt = 0;
        for (int unit = 0; alive && line.next(seg); ++unit) {
            const int most = line_seen(p, seg, seg.rows - 1, S::kRows), least = line_seen(p, seg, 0, S::kRows);
            for (int b = seg.b0; b < seg.b1 && alive; ++b)
                for (int h = 0; h < 2; ++h, ++vt) {
                    const int rs = vt % S::kRawStages, vs = vt % S::kVStages, tok0 = b * kTok + h * kHalf;
                    if (!wait(misc.raw_full[rs], vt / S::kRawStages)) break;
                    if (vt >= S::kVStages && !wait(misc.v_empty[vs], vt / S::kVStages - 1)) break;
                    const uint32_t src = base + S::off_raw + rs * S::kRaw, dst = base + S::off_v + vs * S::kV;
                    const bool end = tok0 + kHalf > most;    // tokens that nobody sees
                    const bool edge = tok0 + kHalf > least;  // tokens that some rows see and others do not
                    constexpr int kChunks = D / 16;          // 16-byte chunks of a row
                    bool poison = false;
#pragma unroll
                    for (int i = 0; i < kHalf * kChunks / 128; ++i) {
                        const int x = i * 128 + t, r = x / kChunks, c = x % kChunks;
                        uint4 v = lds128(src + chunk8_at<D>(kHalf, r, c));
                        if (end && tok0 + r >= most) v = make_uint4(0, 0, 0, 0);
                        if (edge && (has_nan(v.x) || has_nan(v.y) || has_nan(v.z) || has_nan(v.w))) {
                            poison = true;
                            v.x = without_nan(v.x), v.y = without_nan(v.y), v.z = without_nan(v.z), v.w = without_nan(v.w);
                        }
                        const uint32_t row = dst + (c >> 2) * (kHalf * 128) + r * 128;
                        // lanes of the two 64-column blocks write their halves in opposite orders: no bank conflicts
                        const int first = (c >> 2) & 1;
                        const uint32_t a0 = e4m3x2_to_f16x2(v.x), a1 = e4m3x2_to_f16x2(v.x >> 16);
                        const uint32_t a2 = e4m3x2_to_f16x2(v.y), a3 = e4m3x2_to_f16x2(v.y >> 16);
                        const uint32_t b0 = e4m3x2_to_f16x2(v.z), b1 = e4m3x2_to_f16x2(v.z >> 16);
                        const uint32_t b2 = e4m3x2_to_f16x2(v.w), b3 = e4m3x2_to_f16x2(v.w >> 16);
                        const int c0 = (c & 3) * 2;
                        const uint32_t at0 = row + (((c0 + first) ^ (r & 7)) << 4), at1 = row + (((c0 + 1 - first) ^ (r & 7)) << 4);
                        if (first) {
                            sts128(at0, b0, b1, b2, b3);
                            sts128(at1, a0, a1, a2, a3);
                        } else {
                            sts128(at0, a0, a1, a2, a3);
                            sts128(at1, b0, b1, b2, b3);
                        }
                    }
                    if (poison) misc.poison[unit % kPoisonSlots] = unit + 1;
                    tc::fence_async_smem();
                    tc::mbar_arrive(&misc.v_full[vs]);
                    tc::mbar_arrive(&misc.raw_empty[rs]);
                }
        }
    } else {
        // ---- softmax: a query row per thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
        const int group = warp >> 2;  // query tile
        const int row = threadIdx.x & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
        int w = 0;       // items of the CTA so far
        int checked = -1;
        bool bad_pages = false;
        for (int unit = 0; group < NQ && alive && line.next(seg); ++unit) {
            const int tiles = seg.b1 - seg.b0;
            const int r = group * 128 + row, g = seg.tile * S::kRows + r, token = g / p.group;
            const bool real = r < seg.rows;
            const int seen = real ? max(0, seg.kv - seg.count + token + 1) : 0;
            if (checked != seg.seq) {
                bool bad = false;
                const int pages = (seg.kv + p.page - 1) / p.page;
                for (int i = row; i < pages; i += 128) {
                    const int page = p.table[(long long)seg.seq * p.max_pages + i];
                    bad |= page < 0 || page >= p.n_pages;
                }
                bad_pages = softmax_or(group, bad);
                if (bad_pages && row == 0) atomicOr(p.status, SR_DEV_BAD_INDEX);
                checked = seg.seq;
            }
            // the row's query as hi + lo
            float row_scale;
            {
                const __nv_bfloat16 *src =
                    p.q + (long long)(seg.bos + token) * p.q_stride + (seg.head * p.group + g % p.group) * D;
                float top = 0.f;
                if (real)
#pragma unroll 4
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 v = reinterpret_cast<const uint4 *>(src)[c];
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xffff0000u))));
                    }
                const float down = row_down(top) * 256.f;
                row_scale = p.scale_log2 / down;
                const uint32_t hi_at = base + group * 2 * S::kQ, lo_at = hi_at + S::kQ;
#pragma unroll 2
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint4 v = real ? reinterpret_cast<const uint4 *>(src)[2 * c + u] : make_uint4(0, 0, 0, 0);
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float f0 = __uint_as_float(x[2 * e] << 16) * down, f1 = __uint_as_float(x[2 * e] & 0xffff0000u) * down;
                            const float f2 = __uint_as_float(x[2 * e + 1] << 16) * down,
                                        f3 = __uint_as_float(x[2 * e + 1] & 0xffff0000u) * down;
                            const uint32_t h = to_e4m3x4(f0, f1, f2, f3);
                            const float2 a = e4m3x2_to_float2(h), b = e4m3x2_to_float2(h >> 16);
                            hi[2 * u + e] = h;
                            lo[2 * u + e] = to_e4m3x4(f0 - a.x, f1 - a.y, f2 - b.x, f3 - b.y);
                        }
                    }
                    const uint32_t at = chunk8_at<D>(128, row, c);
                    sts128(hi_at + at, hi[0], hi[1], hi[2], hi[3]);
                    sts128(lo_at + at, lo[0], lo[1], lo[2], lo[3]);
                }
                tc::fence_async_smem();
                tc::mbar_arrive(&misc.q_full);
            }

            float m = kNone, l = 0.f;
            const uint32_t o_at = tmem + lanes + 256 + group * 128;
            // lane g of every eight holds the scales of the tile's tokens 16 g .. 16 g + 15, loaded a tile ahead
            auto scales_of = [&](int b, float &ks, float &vs) {
                const int at = b * kTok + (lane & 7) * 16;
                ks = vs = 1.f;
                if (b < seg.b1 && at < seg.kv) {
                    const long long block = (long long)page_at(p, seg.seq, at) * p.h_kv + seg.head;
                    ks = p.k_scale[block], vs = p.v_scale[block];
                }
            };
            float ks_next, vs_next;
            scales_of(seg.b0, ks_next, vs_next);
            for (int t = 0; t < tiles; ++t) {
                const int item = w + t * NQ + group, buf = item & 1;
                const int tok0 = (seg.b0 + t) * kTok;
                const float ks = usable_scale(ks_next), vs = usable_scale(vs_next);
                scales_of(seg.b0 + t + 1, ks_next, vs_next);
                const float lv = log2f(vs), up = 1.f / vs;
                if (!wait(misc.s_full[buf], item >> 1)) break;
                tc::tc_fence_after();
                const uint32_t s_at = tmem + lanes + buf * 128;
                uint32_t x[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tc::tmem_ld_32x32b_x32(s_at + 32 * q, x[q]);
                tc::tmem_ld_wait();
                float top = -INFINITY;
                const bool edge = __any_sync(0xffffffffu, tok0 + kTok > seen);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float k = row_scale * __shfl_sync(0xffffffffu, ks, q), v = __shfl_sync(0xffffffffu, lv, q);
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float s = fmaf(__uint_as_float(x[q >> 1][(q & 1) * 16 + c]), k, v);
                        x[q >> 1][(q & 1) * 16 + c] = __float_as_uint(s);
                    }
                }
                if (edge) {
#pragma unroll
                    for (int c = 0; c < kTok; ++c)
                        if (tok0 + c >= seen) x[c >> 5][c & 31] = __float_as_uint(-INFINITY);
                }
#pragma unroll
                for (int c = 0; c < kTok; ++c) top = fmaxf(top, __uint_as_float(x[c >> 5][c & 31]));
                if (__any_sync(0xffffffffu, top > m + kSlack)) {
                    const float next = fmaxf(m, top), f = exp2f(m - next);
                    m = next, l *= f;
                    if (t > 0) {  // the sums so far, once the product before has added to them
                        if (!wait(misc.pv_done[(item - NQ) & 1], (item - NQ) >> 1)) break;
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t y[32];
                            tc::tmem_ld_32x32b_x32(o_at + c, y);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                            tc::tmem_st_32x32b_x32(o_at + c, y);
                        }
                    }
                }
                const float z = m - kShift;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t y[32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float sum = 0.f;
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const int at = half * 64 + q * 16 + c;
                            const float a = ex2(__uint_as_float(x[at >> 5][at & 31]) - z);
                            const float b = ex2(__uint_as_float(x[at >> 5][(at & 31) + 1]) - z);
                            sum += a + b;
                            y[(q * 16 + c) / 2] = pack_f16(a, b);
                        }
                        l = fmaf(sum, __shfl_sync(0xffffffffu, up, half * 4 + q), l);
                    }
                    tc::tmem_st_32x32b_x32(s_at + 32 * half, y);
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                tc::mbar_arrive(&misc.p_full[buf]);
            }
            const int last = w + (tiles - 1) * NQ + group;
            w += tiles * NQ;
            if (!alive) break;
            if (tiles > 0 && !wait(misc.pv_done[last & 1], last >> 1)) break;
            tc::tc_fence_after();

            // ---- the unit's sums
            const bool whole = seg.first_cta == seg.last_cta;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long out_row = (long long)(seg.bos + token) * p.h_q + seg.head * p.group + g % p.group;
            const int slot = 2 * blockIdx.x + (int(blockIdx.x) == seg.first_cta ? 1 : 0);
            // part sums: [slot][tile][D / 4][128 rows] of four columns, so that neighbouring rows lie together
            float4 *part = reinterpret_cast<float4 *>(p.parts) + (long long)(slot * NQ + group) * (D / 4) * 128 + row;
            const bool poisoned = misc.poison[unit % kPoisonSlots] == unit + 1;
            const int edge0 = line_seen(p, seg, 0, S::kRows) / kHalf * kHalf;  // the first stage that rows see differently
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t y[32];
                if (tiles > 0) {
                    tc::tmem_ld_32x32b_x32(o_at + c, y);
                    tc::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = 0;
                }
                if (poisoned && real && !bad_pages)
                    for (int t = max(edge0, seg.b0 * kTok); t < min(seen, seg.b1 * kTok); ++t) {
                        const uint8_t *v = p.v_cache + (((long long)page_at(p, seg.seq, t) * p.h_kv + seg.head) * p.page + t % p.page) * D + c;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if ((v[e] & 127) == 127) y[e] = 0x7fc00000u;
                    }
                if (whole) {
                    if (real && !bad_pages)
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint4 v;
                            v.x = pack_bf16(__uint_as_float(y[e]) * inv, __uint_as_float(y[e + 1]) * inv);
                            v.y = pack_bf16(__uint_as_float(y[e + 2]) * inv, __uint_as_float(y[e + 3]) * inv);
                            v.z = pack_bf16(__uint_as_float(y[e + 4]) * inv, __uint_as_float(y[e + 5]) * inv);
                            v.w = pack_bf16(__uint_as_float(y[e + 6]) * inv, __uint_as_float(y[e + 7]) * inv);
                            *reinterpret_cast<uint4 *>(p.o + out_row * D + c + e) = v;
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        part[(c + e) / 4 * 128] = make_float4(__uint_as_float(y[e]), __uint_as_float(y[e + 1]),
                                                              __uint_as_float(y[e + 2]), __uint_as_float(y[e + 3]));
                }
            }
            tc::tc_fence_before();
            tc::mbar_arrive(&misc.o_free);
            if (whole) {
                if (real && !bad_pages && p.lse) p.lse[out_row] = log_sum(m, l);
                continue;
            }
            p.part_ml[(slot * NQ + group) * 128 + row] = make_float2(m, l);
            __threadfence();
            softmax_sync(group);
            if (row == 0) {
                int *ticket = &p.tickets[seg.first_cta * NQ + group];
                const bool mine = atomicAdd(ticket, 1) == seg.last_cta - seg.first_cta;
                if (mine) *ticket = 0;
                __threadfence();
                misc.ticket[group] = mine;
            }
            softmax_sync(group);
            if (misc.ticket[group] && real && !bad_pages) {
                const int parts = seg.last_cta - seg.first_cta + 1;
                auto at = [&](int i) { return (2 * (seg.first_cta + i) + (i == 0)) * NQ + group; };
                float M = kNone, L = 0.f;
                for (int i = 0; i < parts; ++i) M = fmaxf(M, __ldcg(&p.part_ml[at(i) * 128 + row]).x);
                for (int i = 0; i < parts; ++i) {
                    const float2 ml = __ldcg(&p.part_ml[at(i) * 128 + row]);
                    L = fmaf(ml.y, exp2f(ml.x - M), L);
                }
                const float one = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 1
                for (int c = 0; c < D / 4; c += 8) {
                    float4 sum[8] = {};
                    for (int i = 0; i < parts; ++i) {
                        const float f = exp2f(__ldcg(&p.part_ml[at(i) * 128 + row]).x - M);
                        const float4 *src = reinterpret_cast<const float4 *>(p.parts) + ((long long)at(i) * (D / 4) + c) * 128 + row;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 v = __ldcg(src + e * 128);
                            sum[e].x = fmaf(f, v.x, sum[e].x), sum[e].y = fmaf(f, v.y, sum[e].y);
                            sum[e].z = fmaf(f, v.z, sum[e].z), sum[e].w = fmaf(f, v.w, sum[e].w);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        *reinterpret_cast<uint4 *>(p.o + out_row * D + 4 * (c + e)) =
                            make_uint4(pack_bf16(sum[e].x * one, sum[e].y * one), pack_bf16(sum[e].z * one, sum[e].w * one),
                                       pack_bf16(sum[e + 1].x * one, sum[e + 1].y * one),
                                       pack_bf16(sum[e + 1].z * one, sum[e + 1].w * one));
                }
                if (p.lse) p.lse[out_row] = log_sum(M, L);
            }
            softmax_sync(group);  // the ticket may be written again
        }
    }
done:
    // a role that gave up leaves copies and products in flight: time for them to end
    if (!alive) __nanosleep(1000000);
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 12) tc::tmem_dealloc(tmem, 512);
}

template <int D> cudaError_t launch(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, cudaStream_t st) {
    const int bytes = PromptSmem<D>::bytes;
    cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    prompt_kernel<D><<<kPromptCtas, kThreads, bytes, st>>>(k, v, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t attend_prompt(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int d, cudaStream_t st) {
    return d == 64 ? launch<64>(k, v, p, st) : d == 128 ? launch<128>(k, v, p, st) : launch<256>(k, v, p, st);
}

}  // namespace paged
}  // namespace sr
