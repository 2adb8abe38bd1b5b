// Appending keys and values to a paged 8-bit cache, with the position rotation
// of queries and keys on the way.
//
// Per token, head and rotated pair i, with the angle f = position * inv_freq[i]
// of the axis that pair i belongs to: (lo, hi) -> (lo cos f - hi sin f,
// lo sin f + hi cos f).  A page of a head is a block with one power-of-two
// scale s; a value x is stored as e4m3(x / s), so storing and reading back cost
// one rounding and no other.  Where new tokens join older ones in a page, the
// page keeps the larger of its scale and what the new ones need, and the older
// bytes are rounded again if it grew (dividing by a power of two is exact, so
// only values that fall into e4m3's least binade change).
//
// Bound by memory: queries 2 + 2 bytes a value, keys and values 2 + 1.  One
// CTA per page of a sequence's new tokens (and per share of the heads): it
// forms the page's cosines and sines once, in shared memory, for all its heads,
// since an angle (64-bit product, reduced to a fraction of a turn, because a
// position of 10^6 times 1 rad leaves fp32 no fraction) costs more than the
// rotation itself.  A warp takes one head of the page: keys and values in two
// passes over the bf16 rows, the first for the largest magnitude, the second
// from the caches that the first filled.  Measured: 8917 new tokens of eight
// requests, 32 + 8 heads of 128, positions on three axes, 55 us (3.8 TB/s on the
// bytes that have to move); one token for each of 64 requests, 16 + 4 heads of
// 256, 6 us a call in a captured graph.
#include <type_traits>

#include "paged.cuh"

namespace sr {
namespace {

constexpr int kWarps = 8;
constexpr double kTurnsPerRadian = 0.15915494309189533577;  // 1 / (2 pi)

struct AppendParams {
    const __nv_bfloat16 *k, *v, *q;
    __nv_bfloat16 *q_out;
    const int32_t *positions;  // [axes, T] or null
    const float *inv_freq;     // [rot / 2]
    const int32_t *cu, *kv_lens, *table;
    uint8_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
    uint32_t *status;
    long long k_stride, v_stride, q_stride, q_out_stride;
    int n_seqs, total, max_len, h_q, h_kv, page, n_pages, max_pages, half, interleaved, sec0, sec1, groups;
};

// Eight elements of a token's head that one lane holds: four rotated pairs
// (4u .. 4u+3) for u < half / 4, eight elements without rotation beyond.
struct Unit {
    int lo, hi;   // element offsets of the two 4-element parts
    int pair;     // first pair, or -1
};

template <int D>
__device__ __forceinline__ Unit unit_of(int u, int half, int interleaved) {
    Unit r;
    if (u < half / 4) {
        r.pair = 4 * u;
        r.lo = interleaved ? 8 * u : 4 * u;
        r.hi = interleaved ? 8 * u + 4 : half + 4 * u;
    } else {
        r.pair = -1;
        r.lo = 8 * u;
        r.hi = 8 * u + 4;
    }
    return r;
}

__device__ __forceinline__ void unpack(uint2 r, float *f) {
    f[0] = __uint_as_float(r.x << 16);
    f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16);
    f[3] = __uint_as_float(r.y & 0xffff0000u);
}

// f[0..3] at u.lo, f[4..7] at u.hi.  Lanes without pairs keep what they have by selection: a branch would keep the
// tokens of a batch from overlapping, and a product with (1, 0) would spread what is not finite.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&f)[8], const Unit &u, const float2 *cs, int half) {
    // a token's cosines and sines: pairs 4u, 4u+1 of every u, then 4u+2, 4u+3, so that lanes read neighbouring 16 bytes
    const float2 *at = cs + max(u.pair, 0) / 2;
    const float4 one = *reinterpret_cast<const float4 *>(at), two = *reinterpret_cast<const float4 *>(at + half / 2);
    const float2 cc[4] = {{one.x, one.y}, {one.z, one.w}, {two.x, two.y}, {two.z, two.w}};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 c = cc[j];
        float &lo = INTER ? f[2 * j] : f[j], &hi = INTER ? f[2 * j + 1] : f[4 + j];
        const float x = lo * c.x - hi * c.y, y = lo * c.y + hi * c.x;
        lo = u.pair < 0 ? lo : x;
        hi = u.pair < 0 ? hi : y;
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(AppendParams p) {
    constexpr int kLanes = D / 8;         // lanes per token
    constexpr int kAtOnce = 32 / kLanes;  // tokens per warp and step
    constexpr int kBatch = 4;             // steps whose rows are loaded together
    extern __shared__ __align__(16) float2 table_cs[];  // [tokens of the page][half], in rotate's order
    const int seq = blockIdx.z;
    int bos, eos;
    if (!seq_bounds(p.cu, seq, p.total, p.max_len, p.status, bos, eos)) return;
    if (bos == eos) return;
    const int kv = p.kv_lens[seq], start = kv - (eos - bos);
    if (start < 0 || kv > (long long)p.max_pages * p.page) {
        if (threadIdx.x == 0) atomicOr(p.status, SR_DEV_BAD_LENGTH);
        return;
    }
    const int slot = start / p.page + blockIdx.x;  // page of the sequence
    const int from = max(start, slot * p.page), to = min(kv, (slot + 1) * p.page);
    if (from >= to) return;
    const int n = to - from, tok0 = bos + (from - start);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    for (int i = threadIdx.x; i < n * p.half; i += kWarps * 32) {
        const int t = i / p.half, pair = i - t * p.half;
        const int axis = (pair >= p.sec0) + (pair >= p.sec1);
        const long long at = (long long)axis * p.total + tok0 + t;
        const int pos = !p.positions ? from + t : SR_IN_BOUNDS(at, 3ll * p.total, p.status) ? p.positions[at] : 0;
        const double turns = double(pos) * double(p.inv_freq[pair]) * kTurnsPerRadian;
        float s, c;
        sincospif(2.f * float(turns - rint(turns)), &s, &c);
        table_cs[t * p.half + (pair & 2) / 2 * (p.half / 2) + pair / 4 * 2 + (pair & 1)] = make_float2(c, s);
    }
    __syncthreads();

    const int page = p.table[(long long)seq * p.max_pages + slot];
    const bool page_ok = page >= 0 && page < p.n_pages;
    if (!page_ok && threadIdx.x == 0) atomicOr(p.status, SR_DEV_BAD_INDEX);
    const Unit u = unit_of<D>(lane % kLanes, p.half, INTER);
    const Unit plain{8 * (lane % kLanes), 8 * (lane % kLanes) + 4, -1};
    const int sub = lane / kLanes;
    // Calls use(t, f) for every token t of this lane, f being its eight elements; with `turn`, rotated.
    auto walk = [&](const __nv_bfloat16 *src, long long stride, const Unit &w, auto turn, auto use) {
#pragma unroll 1
        for (int t0 = 0; t0 < n; t0 += kBatch * kAtOnce) {
            uint2 in[kBatch][2];  // behind the last token: the last once more, to the same result
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int t = min(t0 + sub + i * kAtOnce, n - 1);
                const __nv_bfloat16 *row = src + t * stride;
                in[i][0] = in[i][1] = make_uint2(0, 0);
                if (!SR_IN_BOUNDS(tok0 + t, p.total, p.status)) continue;
                in[i][0] = *reinterpret_cast<const uint2 *>(row + w.lo);
                in[i][1] = *reinterpret_cast<const uint2 *>(row + w.hi);
            }
            __syncwarp();  // in place, every copy of a row is read before the first is written
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int t = min(t0 + sub + i * kAtOnce, n - 1);
                float f[8];
                unpack(in[i][0], f);
                unpack(in[i][1], f + 4);
                if (turn) rotate<INTER>(f, w, table_cs + t * p.half, p.half);
                use(t, f);
            }
        }
    };
    const int heads = p.h_q + 2 * p.h_kv;
    for (int item = blockIdx.y * kWarps + warp; item < heads; item += p.groups * kWarps) {
        if (item >= 2 * p.h_kv) {  // a query head: rotated rows
            const int h = item - 2 * p.h_kv;
            __nv_bfloat16 *dst = p.q_out + (long long)tok0 * p.q_out_stride + h * D;
            walk(p.q + (long long)tok0 * p.q_stride + h * D, p.q_stride, u, std::true_type{}, [&](int t, const float(&f)[8]) {
                __nv_bfloat16 *out = dst + t * p.q_out_stride;
                if (!SR_IN_BOUNDS(tok0 + t, p.total, p.status)) return;
                *reinterpret_cast<uint2 *>(out + u.lo) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
                *reinterpret_cast<uint2 *>(out + u.hi) = make_uint2(pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
            });
            continue;
        }
        if (!page_ok || !SR_IN_BOUNDS(slot, p.max_pages, p.status)) continue;
        const bool key = item < p.h_kv;
        const int h = key ? item : item - p.h_kv;
        const Unit w = key ? u : plain;
        const long long stride = key ? p.k_stride : p.v_stride;
        const __nv_bfloat16 *src = (key ? p.k : p.v) + (long long)tok0 * stride + h * D;
        const long long block = (long long)page * p.h_kv + h;
        uint8_t *cache = (key ? p.k_cache : p.v_cache) + block * p.page * D;
        float *scale = (key ? p.k_scale : p.v_scale) + block;
        float top = 0.f;
        auto largest = [&](int, const float(&f)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = fabsf(f[j]);
                top = fmaxf(top, m <= 3.402823466e38f ? m : 0.f);  // what is not finite has no part in the scale
            }
        };
        if (key) walk(src, stride, w, std::true_type{}, largest); else walk(src, stride, w, std::false_type{}, largest);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int old = from - slot * p.page;  // tokens that the page held before
        const float before = old > 0 ? *scale : 0.f;
        const float kept = fmaxf(before, ldexpf(1.f, paged::scale_exp(top)));
        __syncwarp();  // every lane has read the old scale
        if (lane == 0) *scale = kept;
        if (old > 0 && before != kept) {
            const float ratio = before / kept;
            for (int t = sub; t < old; t += kAtOnce) {
                uint2 *at = reinterpret_cast<uint2 *>(cache + t * D + plain.lo);
                uint2 r = *at;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t &x = j ? r.y : r.x;
                    const float2 a = paged::e4m3x2_to_float2(x), b = paged::e4m3x2_to_float2(x >> 16);
                    x = paged::to_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
                }
                *at = r;
            }
        }
        const float inv = 1.f / kept;
        auto store = [&](int t, const float(&f)[8]) {
            uint8_t *out = cache + (old + t) * D;
            if (!SR_IN_BOUNDS(old + t, p.page, p.status)) return;
            *reinterpret_cast<uint32_t *>(out + w.lo) = paged::to_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
            *reinterpret_cast<uint32_t *>(out + w.hi) = paged::to_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
        };
        if (key) walk(src, stride, w, std::true_type{}, store); else walk(src, stride, w, std::false_type{}, store);
    }
}

template <int D, bool INTER>
cudaError_t launch(AppendParams p, cudaStream_t st) {
    const int slots = (p.max_len + p.page - 2) / p.page + 1;  // pages that max_len tokens can touch
    const int heads = (p.q ? p.h_q : 0) + 2 * p.h_kv;
    // The heads of a page are shared out over as many CTAs as give the GPU eight warps per scheduler; every share
    // repeats the page's cosines and sines, so no more than that.
    // pages that there can be: of the longest sequences, and of all tokens with a part page at both ends
    const long long most_tiles = (long long)slots * p.n_seqs, full = p.total / p.page + 2ll * p.n_seqs;
    const long long tiles = most_tiles < full ? most_tiles : full;
    const int most = (heads + kWarps - 1) / kWarps;
    const long long want = (4 * 148 + tiles - 1) / tiles;
    const int rounds = want < most ? int((most + want - 1) / want) : 1;  // heads of a warp, the same for all
    p.groups = (most + rounds - 1) / rounds;
    // Four entries at least: lanes without pairs (all of them without a rotation) read the first four of a token's, and
    // keep what they have.
    const size_t entries = size_t(p.page < p.max_len ? p.page : p.max_len) * p.half;
    const size_t smem = (entries > 4 ? entries : 4) * sizeof(float2);
    static_assert(128 * 128 * sizeof(float2) <= 227 * 1024, "the largest table fits");
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(append_kernel<D, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
    }
    append_kernel<D, INTER><<<dim3(slots, p.groups, p.n_seqs), kWarps * 32, smem, st>>>(p);
    return cudaGetLastError();
}

template <bool INTER> cudaError_t pick(const AppendParams &p, int d, cudaStream_t st) {
    return d == 64 ? launch<64, INTER>(p, st) : d == 128 ? launch<128, INTER>(p, st) : launch<256, INTER>(p, st);
}

sr_status validate(const sr_kv_append_args *a) {
    if (!a) return set_error(SR_ERR_INVALID_ARG, "args is NULL");
    if (sr_status s = check_varlen(a->n_seqs, a->total_tokens, a->max_seqlen, a->cu_seqlens)) return s;
    if (a->total_tokens > (1 << 30)) return set_error(SR_ERR_UNSUPPORTED, "total_tokens > 2^30");
    if (sr_status s = check_cache(a->n_pages, a->max_pages, a->page_size, a->h_q, a->h_kv, a->head_dim, a->q != nullptr))
        return s;
    if (!a->k || !a->v || !a->kv_lens || !a->block_table || !a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale)
        return set_error(SR_ERR_INVALID_ARG, "k, v, kv_lens, block_table, caches and scales are required");
    if (!a->q != !a->q_out) return set_error(SR_ERR_INVALID_ARG, "q and q_out come together");
    if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 8)
        return set_error(SR_ERR_UNSUPPORTED, "rot_dim must be a multiple of 8 in 0..head_dim (got %d)", a->rot_dim);
    if (a->rot_dim > 0 && !a->inv_freq) return set_error(SR_ERR_INVALID_ARG, "inv_freq is required with rot_dim > 0");
    if (a->n_axes < 1 || a->n_axes > 3) return set_error(SR_ERR_UNSUPPORTED, "n_axes must be 1, 2 or 3");
    int sum = 0;
    for (int i = 0; i < a->n_axes; ++i) {
        if (a->sections[i] < 0 || a->sections[i] > a->rot_dim)
            return set_error(SR_ERR_INVALID_ARG, "sections[%d] is out of range", i);
        sum += a->sections[i];
    }
    if (sum != a->rot_dim / 2) return set_error(SR_ERR_INVALID_ARG, "sections must add up to rot_dim / 2");
    if (a->n_axes > 1 && !a->positions) return set_error(SR_ERR_INVALID_ARG, "several axes need positions");
    const struct { const void *p; int64_t stride; int heads; const char *name; } rows[] = {
        {a->k, a->k_stride, a->h_kv, "k"}, {a->v, a->v_stride, a->h_kv, "v"},
        {a->q, a->q_stride, a->h_q, "q"}, {a->q_out, a->q_out_stride, a->h_q, "q_out"}};
    for (const auto &r : rows)
        if (r.p && (r.stride < int64_t(r.heads) * a->head_dim || r.stride % 8 || !aligned(r.p, 16)))
            return set_error(SR_ERR_INVALID_ARG, "%s: 16-byte aligned, its token stride a multiple of 8 and no less than "
                             "a token's heads", r.name);
    if (!aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !aligned(a->k_scale, 4) || !aligned(a->v_scale, 4))
        return set_error(SR_ERR_INVALID_ARG, "caches must be 16-byte aligned, scales 4-byte");
    return SR_OK;
}

}  // namespace

sr_status check_cache(int n_pages, int max_pages, int page, int h_q, int h_kv, int d, bool queries) {
    if (n_pages < 0 || max_pages < 0) return set_error(SR_ERR_INVALID_ARG, "negative n_pages or max_pages");
    if (page != 16 && page != 32 && page != 64 && page != 128)
        return set_error(SR_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128 (got %d)", page);
    if (d != 64 && d != 128 && d != 256)
        return set_error(SR_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", d);
    if (h_kv <= 0 || (queries && (h_q <= 0 || h_q % h_kv)))
        return set_error(SR_ERR_INVALID_ARG, "need h_kv > 0 and h_q a multiple of it (h_q=%d h_kv=%d)", h_q, h_kv);
    if (h_kv > 1024 || h_q > 4096) return set_error(SR_ERR_UNSUPPORTED, "h_kv > 1024 or h_q > 4096");
    if ((long long)max_pages * page > (1 << 30))
        return set_error(SR_ERR_UNSUPPORTED, "max_pages * page_size > 2^30");
    return SR_OK;
}

}  // namespace sr

using namespace sr;

extern "C" size_t sr_kv_append_workspace(const sr_kv_append_args *a) { return validate(a) ? 0 : kWsHeader; }

extern "C" sr_status sr_kv_append(const sr_kv_append_args *a, void *ws, size_t ws_bytes, void *stream) {
    if (sr_status s = validate(a)) return s;
    if (sr_status s = check_workspace(ws, ws_bytes, kWsHeader)) return s;
    AppendParams p{};
    p.k = static_cast<const __nv_bfloat16 *>(a->k), p.v = static_cast<const __nv_bfloat16 *>(a->v);
    p.q = static_cast<const __nv_bfloat16 *>(a->q), p.q_out = static_cast<__nv_bfloat16 *>(a->q_out);
    p.positions = a->positions, p.inv_freq = a->inv_freq;
    p.cu = a->cu_seqlens, p.kv_lens = a->kv_lens, p.table = a->block_table;
    p.k_cache = static_cast<uint8_t *>(a->k_cache), p.v_cache = static_cast<uint8_t *>(a->v_cache);
    p.k_scale = a->k_scale, p.v_scale = a->v_scale;
    p.status = static_cast<uint32_t *>(ws);
    p.k_stride = a->k_stride, p.v_stride = a->v_stride, p.q_stride = a->q_stride, p.q_out_stride = a->q_out_stride;
    p.n_seqs = a->n_seqs, p.total = a->total_tokens, p.max_len = a->max_seqlen;
    p.h_q = a->q ? a->h_q : 0, p.h_kv = a->h_kv, p.page = a->page_size, p.n_pages = a->n_pages;
    p.max_pages = a->max_pages, p.half = a->rot_dim / 2, p.interleaved = a->interleaved != 0;
    p.sec0 = a->n_axes > 1 ? a->sections[0] : p.half;
    p.sec1 = a->n_axes > 2 ? a->sections[0] + a->sections[1] : p.half;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(p.status, 0, sizeof(uint32_t), st);
    if (e == cudaSuccess && p.n_seqs > 0 && p.max_len > 0)
        e = p.interleaved ? pick<true>(p, a->head_dim, st) : pick<false>(p, a->head_dim, st);
    return e == cudaSuccess ? SR_OK : cuda_error(e, "sr_kv_append");
}
