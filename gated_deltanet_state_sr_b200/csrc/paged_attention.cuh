// What the kernels of attention over the paged 8-bit cache share.
#pragma once

#include <cuda.h>

#include "paged.cuh"
#include "tc.cuh"

namespace sr {
namespace paged {

struct AttnParams {
    const __nv_bfloat16 *q;
    long long q_stride;  // elements from token to token
    const int32_t *cu, *kv_lens, *table;
    const float *k_scale, *v_scale;
    const uint8_t *v_cache;
    __nv_bfloat16 *o;
    float *lse;  // may be null
    uint32_t *status;
    int *tickets;     // zero at the start of a call
    float *parts;     // partial O
    float2 *part_ml;  // their m and l
    float scale_log2; // scale log2(e)
    int n_seqs, total, max_len, max_kv, h_q, h_kv, group, page, n_pages, max_pages;
};

// Both kernels run one CTA per SM.
constexpr int kRowsMaxCtas = 148, kPromptCtas = 148;
// Rows of a partial sum, and their number: two for every CTA, the end of one unit and the beginning of another.
constexpr int prompt_rows(int d) { return d == 256 ? 128 : 256; }

constexpr float kNone = -1e30f;  // m of a row that has seen nothing
constexpr float kSlack = 4.f;    // growth of the maximum that m does not follow
constexpr float kShift = 11.f;   // weights are at most 2^(kShift + kSlack) = 2^15

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Power of two that brings a row whose largest element is `top` to at most 1.
__device__ __forceinline__ float row_down(float top) {
    if (!(top > 0.f) || top > 3.402823466e38f) return 1.f;
    int e;
    frexpf(top, &e);
    return ldexpf(1.f, -min(max(e, -100), 120));
}
// A block's scale, within the range that sr_kv_append writes; NaN becomes the least.
__device__ __forceinline__ float usable_scale(float s) { return fminf(fmaxf(s, 0x1p-32f), 0x1p32f); }
// log(sum exp(s)) of a row from its base-2 m and l.
__device__ __forceinline__ float log_sum(float m, float l) {
    return l == 0.f ? -INFINITY : 0.69314718055994531f * (m - kShift + log2f(l));
}
// e4m3 NaN bytes (0x7f, 0xff) of a word.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ bool has_nan(uint32_t w) { return nan_bits(w) != 0; }
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~((nan_bits(w) >> 7) * 0xffu); }

// The work of a call as one line of blocks, of which every CTA takes an equal
// part.  A unit is ROWS query rows (row = token * group + head of the group) of a
// (sequence, key/value head); it has one block for every TOK cached tokens that
// its last row sees (one at least: rows that see nothing are written too).
// Units of a sequence follow one another head by head, tile by tile.
struct Segment {
    int seq, head, tile, rows;   // rows: of this tile
    int b0, b1, blocks;          // this CTA's blocks of the unit, and how many it has
    int bos, count, kv;          // the sequence: first row, new tokens, cached tokens
    int first_cta, last_cta;     // CTAs that hold the unit's blocks
};

struct LinePlace {
    long long scan[32], at;
    int seq;
};

template <int ROWS, int TOK> struct Line {
    const AttnParams *p;
    long long cur, end, total;
    int ctas, seq, bos, count, kv, tiles, head, tile, block;

    __device__ __forceinline__ int seen_by(int r) const {  // tokens that the last row of tile r sees
        const int last = min((r + 1) * ROWS, count * p->group) - 1;
        return max(0, kv - count + last / p->group + 1);
    }
    __device__ __forceinline__ int blocks_of(int r) const { return max(1, (seen_by(r) + TOK - 1) / TOK); }

    // Sequence n; the blocks of one of its heads, 0 where its entries are out of range (or it has no rows).
    __device__ long long load(int n, bool flag) {
        int b = p->cu[n], e = p->cu[n + 1], k = p->kv_lens[n];
        uint32_t bad = 0;
        if (b < 0 || b > e || e > p->total || (n == 0 && b != 0)) bad = SR_DEV_BAD_CU_SEQLENS;
        else if (e - b > p->max_len) bad = SR_DEV_SEQ_TOO_LONG;
        else if (k < 0 || k > p->max_kv || k > (long long)p->max_pages * p->page) bad = SR_DEV_BAD_LENGTH;
        if (bad) {
            if (flag) atomicOr(p->status, bad);
            e = b, k = 0;
        }
        bos = b, count = e - b, kv = k;
        tiles = (count * p->group + ROWS - 1) / ROWS;
        long long sum = 0;
        for (int r = 0; r < tiles; ++r) sum += blocks_of(r);
        return sum;
    }

    // Finds the part of this CTA; all `THREADS` threads of the block call it.  False: there is none.
    template <int THREADS> __device__ bool start(const AttnParams &params, int min_blocks, LinePlace &place) {
        p = &params;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        long long mine = 0;
        for (int n = threadIdx.x; n < p->n_seqs; n += THREADS) mine += load(n, blockIdx.x == 0) * p->h_kv;
#pragma unroll
        for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        if (lane == 0) place.scan[warp] = mine;
        __syncthreads();
        total = 0;
        for (int w = 0; w < THREADS / 32; ++w) total += place.scan[w];
        if (total == 0) return false;
        ctas = int(min((long long)gridDim.x, (total + min_blocks - 1) / min_blocks));
        if (int(blockIdx.x) >= ctas) return false;
        cur = blockIdx.x * total / ctas;
        end = (blockIdx.x + 1) * total / ctas;
        // the sequence that holds block `cur`: sums over THREADS sequences at a time
        long long before = 0;
        for (int n0 = 0; before <= cur; n0 += THREADS) {
            const int n = n0 + threadIdx.x;
            const long long c = n < p->n_seqs ? load(n, false) * p->h_kv : 0;
            long long incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            __syncthreads();
            if (lane == 31) place.scan[warp] = incl;
            __syncthreads();
            long long at = before + incl - c, chunk = 0;
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w < warp) at += place.scan[w];
                chunk += place.scan[w];
            }
            if (c > 0 && cur >= at && cur < at + c) place.seq = n, place.at = at;
            before += chunk;
        }
        __syncthreads();
        seq = place.seq;
        const long long per_head = load(seq, false);
        long long local = cur - place.at;
        head = int(local / per_head);
        local -= head * per_head;
        for (tile = 0; local >= blocks_of(tile); ++tile) local -= blocks_of(tile);
        block = int(local);
        return true;
    }

    __device__ bool next(Segment &s) {
        if (cur >= end) return false;
        const int blocks = blocks_of(tile);
        const int n = int(min((long long)(blocks - block), end - cur));
        s.seq = seq, s.head = head, s.tile = tile;
        s.rows = min(ROWS, count * p->group - tile * ROWS);
        s.b0 = block, s.b1 = seen_by(tile) > 0 ? block + n : block, s.blocks = blocks;
        s.bos = bos, s.count = count, s.kv = kv;
        const long long first = cur - block;
        s.first_cta = int(((first + 1) * ctas - 1) / total);
        s.last_cta = int(((first + blocks) * ctas - 1) / total);
        cur += n;
        block += n;
        if (block == blocks) {
            block = 0;
            if (++tile == tiles) {
                tile = 0;
                if (++head == p->h_kv) {
                    head = 0;
                    if (cur < end)
                        while (load(++seq, false) == 0) {
                        }
                }
            }
        }
        return true;
    }
};

// Tokens that row r of a segment's tile sees.
__device__ __forceinline__ int line_seen(const AttnParams &p, const Segment &s, int r, int rows) {
    return max(0, s.kv - s.count + (s.tile * rows + r) / p.group + 1);
}

// D[tmem] (+)= A[tmem] * B[smem]^T, kind::f16 with half-precision operands (see tc::mma_bf16_ts).
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    tc::mma_bf16_ts(d_tmem, a_tmem, b_desc, idesc, accumulate);  // the types are the descriptor's
}

cudaError_t attend_prompt(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int d, cudaStream_t st);
cudaError_t attend_rows(const CUtensorMap &k, const CUtensorMap &v, const AttnParams &p, int d, cudaStream_t st);

}  // namespace paged
}  // namespace sr
