// embed.hip -- the dense token embedding beside the hashed tables: rows of a
// [vocab][d] table scaled into the hidden state of every residual branch, and
// the table's gradient by sorted tokens.
//
// Forward: h[m][t] = round(scale * table[id_t]), a row copy bound by memory
// (32,768 x 2560 bf16: 64 us, 5.2 TB/s counting every row once in and out).
//
// Backward: dtable[r] = scale * sum over {t : id_t = r} (ascending) and
// branches m of dh[m][t], with no float atomics: the results depend on the
// inputs alone.  Up to 512 tokens one launch does it all (embed_few_kernel);
// beyond that three:
//   embed_sort_kernel   stable counting sort of the token positions by id;
//                       beside it the table's first rows are filled with zeros.
//   embed_rows_kernel   sums of the runs inside each chunk of sorted
//                       positions; zeros for the other rows without tokens.
//   embed_join_kernel   runs that cross chunks, from the chunks' parts.
// The zeros are most of the bytes (4 * vocab * d).  The sort is a latency chain
// of about 20 us, which kFillBeside of them hide.  Measured with a table of
// 129,280 x 2560, 32,768 tokens and four branches: 411 us; all zeros beside the
// sort, which writes the rows with tokens twice, 424; none there 432.  The sums
// and zeros together move 5.3 TB/s, a large copy's rate.
#include <algorithm>

#include "engram_internal.h"
#include "vec8.h"

namespace engram {
namespace {

// One wave per (token, 512 channels): 8 channels a lane.
template <typename T>
__global__ __launch_bounds__(256) void embed_kernel(const int32_t *tokens, int64_t n_tok, int32_t vocab,
                                                    const T *table, int32_t d, int32_t n_branches, float scale,
                                                    T *h, uint32_t *bad) {
    const int lane = threadIdx.x & 63;
    const int32_t strips = (d + 511) / 512;
    const int64_t waves = (int64_t)gridDim.x * 4, n_items = n_tok * strips;
    for (int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); item < n_items; item += waves) {
        const int64_t t = quotient(item, strips);
        const int32_t strip = (int32_t)(item - t * strips);
        const int32_t c = strip * 512 + lane * 8;
        const int32_t id = tokens[t];
        const bool ok = id >= 0 && id < vocab;
        if (!ok && strip == 0 && lane == 0 && bad) atomicAdd(bad, 1u);
        if (c >= d) continue;
        F8 x = {};
        if (ok) {
            x = load8(table + (int64_t)id * d + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) x.v[i] *= scale;
        }
        for (int m = 0; m < n_branches; ++m) store8(h + ((int64_t)m * n_tok + t) * d + c, x);
    }
}

// Stable counting sort by id in one launch: a workgroup owns a bucket of ids
// [b * kBucket, (b + 1) * kBucket) and one of `parts` pieces of the tokens, and
// reads every token (they stay in L2).  First pass: how many tokens have a
// lower id (where the bucket's output starts; no workgroup waits for another),
// how many of each id lie in the pieces before and behind its own, and a count
// per id and wave of its own piece.  Second pass: wave w places the tokens of
// its share of the piece in order, 64 at a time, equal ids ranked by a ballot
// per bit of the id's place in the bucket.  The cost is n_tok * (vocab /
// kBucket) * parts id reads; the placement, most of the time where buckets are
// few, is shared by the parts.
constexpr int kSortWaves = 16;
constexpr int kBucketBits = 9;
constexpr int kBucket = 1 << kBucketBits;

// Bytes of the table that a block of the fill clears.
constexpr int64_t kFillBytes = (int64_t)64 * kSortWaves * 16 * 16;
constexpr int64_t kFillBeside = (int64_t)256 << 20;  // most bytes filled beside the sort

__global__ __launch_bounds__(64 * kSortWaves) void embed_sort_kernel(const int32_t *tokens, int64_t n_tok,
                                                                     int32_t vocab, uint32_t *order, int32_t *sid,
                                                                     uint32_t *start, uint32_t sort_blocks, int32_t parts,
                                                                     float *dtable, int64_t fill_bytes) {
    __shared__ uint32_t cnt[kSortWaves][kBucket];
    __shared__ uint32_t ahead[kBucket], behind[kBucket];  // of each id, in the pieces before and behind
    __shared__ uint32_t below_s[kSortWaves], wtot[kBucket / 64];
    if (blockIdx.x >= sort_blocks) {
        const int64_t at = (int64_t)(blockIdx.x - sort_blocks) * kFillBytes;
        char *dst = reinterpret_cast<char *>(dtable) + at;
        const int64_t n = min(kFillBytes, fill_bytes - at);
        for (int64_t o = threadIdx.x * 16; o < n; o += 64 * kSortWaves * 16)
            *reinterpret_cast<f32x4_t *>(dst + o) = f32x4_t{0.f, 0.f, 0.f, 0.f};
        return;
    }
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const uint32_t bucket = blockIdx.x / (uint32_t)parts, piece = blockIdx.x - bucket * (uint32_t)parts;
    const int64_t lo64 = (int64_t)bucket * kBucket;
    const int32_t lo = (int32_t)lo64;
    const int32_t n_ids = (int32_t)min((int64_t)kBucket, (int64_t)vocab - lo64);
    for (int i = threadIdx.x; i < kSortWaves * kBucket; i += 64 * kSortWaves) (&cnt[0][0])[i] = 0u;
    if (threadIdx.x < kBucket) ahead[threadIdx.x] = behind[threadIdx.x] = 0u;
    __syncthreads();
    const int64_t per = (int64_t)64 * kSortWaves * parts, share = (n_tok + per - 1) / per * 64;
    const int64_t p0 = min(piece * kSortWaves * share, n_tok), p1 = min(p0 + kSortWaves * share, n_tok);
    const int64_t first = min(p0 + w * share, p1), last = min(first + share, p1);
    uint32_t below = 0u;
    int32_t id[8];
    for (int64_t g = w * (64 * 8); g < n_tok - (p1 - p0); g += kSortWaves * (64 * 8)) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t i = g + 64 * u + lane, t = i < p0 ? i : i + (p1 - p0);
            id[u] = t < n_tok ? tokens[t] : -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            below += (id[u] >= 0 && id[u] < lo) ? 1u : 0u;
            if (id[u] >= lo && id[u] - lo < n_ids)
                atomicAdd((g + 64 * u + lane < p0 ? ahead : behind) + (id[u] - lo), 1u);
        }
    }
    for (int64_t g = first; g < last; g += 64 * 8) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t t = g + 64 * u + lane;
            id[u] = t < last ? tokens[t] : -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            below += (id[u] >= 0 && id[u] < lo) ? 1u : 0u;
            if (id[u] >= lo && id[u] - lo < n_ids) atomicAdd(&cnt[w][id[u] - lo], 1u);
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) below += __shfl_xor(below, off);
    if (lane == 0) below_s[w] = below;
    __syncthreads();
    // exclusive prefix over the ids (thread r: id lo + r), then over the waves of each id
    const int r = threadIdx.x;
    uint32_t base = 0u, tot = 0u, incl = 0u;
    for (int i = 0; i < kSortWaves; ++i) base += below_s[i];
    if (r < kBucket) {
        tot = ahead[r] + behind[r];
        for (int i = 0; i < kSortWaves; ++i) tot += cnt[i][r];
        incl = tot;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const uint32_t y = __shfl_up(incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 63) wtot[w] = incl;
    }
    __syncthreads();
    if (r < kBucket) {
        uint32_t at = base + incl - tot;
        for (int i = 0; i < w; ++i) at += wtot[i];
        if (piece == 0u) {
            if (r < n_ids) start[lo + r] = at;
            if (lo64 + r == (int64_t)vocab - 1) start[vocab] = at + tot;
        }
        at += ahead[r];
        for (int i = 0; i < kSortWaves; ++i) {
            const uint32_t c = cnt[i][r];
            cnt[i][r] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t g = first; g < last; g += 64 * 8) {
        if (share > 64 * 8) {  // (else the first pass left them in id)
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t t = g + 64 * u + lane;
                id[u] = t < last ? tokens[t] : -1;
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool mine = id[u] >= lo && id[u] - lo < n_ids;
            uint64_t peers = __ballot(mine);
            if (peers == 0ull) continue;
            const uint32_t at = mine ? (uint32_t)(id[u] - lo) : 0u;
#pragma unroll
            for (int bit = 0; bit < kBucketBits; ++bit) {
                const bool set = ((at >> bit) & 1u) != 0u;
                const uint64_t m = __ballot(set);
                peers &= set ? m : ~m;
            }
            if (mine) {
                const uint32_t pos = cnt[w][at] + (uint32_t)__popcll(peers & ((1ull << lane) - 1ull));
                order[pos] = (uint32_t)(g + 64 * u + lane);
                sid[pos] = id[u];
                // (a wave's LDS accesses complete in order: every peer has read the slot)
                asm volatile("" ::: "memory");
                if ((peers >> lane) == 1ull) cnt[w][at] = pos + 1u;
            }
            asm volatile("" ::: "memory");
        }
    }
}

__device__ __forceinline__ void put_row(float *dst, const F8 &acc, float scale, bool accumulate) {
    F8 x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.v[i] = acc.v[i] * scale;
    if (accumulate) {
        const F8 old = load8(dst);
#pragma unroll
        for (int i = 0; i < 8; ++i) x.v[i] += old.v[i];
    }
    store8(dst, x);
}

// Up to kFew tokens: the gradient in one launch, whose three would each be no
// longer than their launch.  A wave per (token, 512 channels) finds the tokens
// of the same id by ballot, leaves if one comes before, and adds all of them
// in order.  Blocks from sum_blocks on write zeros to the rows without tokens.
// What bounds it is the longest run, one wave's chain of trips to memory with U
// tokens each: 512 tokens of 1000 x 1024 in bf16 with one branch and with four
// take 6.4 and 6.3 us if all differ, 10.2 and 23.5 by a Zipf law, 50 and 169 if
// all are one id; sorted (513 of them) 12.6 and 13.8, 13.7 and 14.9, 13.2 and 14.5.
constexpr int kFew = 512;

template <typename T, int BR>
__global__ __launch_bounds__(256) void embed_few_kernel(const int32_t *tokens, int32_t n_tok, int32_t vocab, int32_t d,
                                                        const T *dh, float scale, bool accumulate, float *dtable,
                                                        uint32_t sum_blocks) {
    constexpr int U = BR <= 2 ? 8 : 4;
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (blockIdx.x >= sum_blocks) {
        const int64_t r0 = (wave - (int64_t)sum_blocks * 4) * 8;
        uint32_t named = 0u;  // bit k: row r0 + k has a token
        for (int32_t g = 0; g < n_tok; g += 64) {
            const int64_t k = g + lane < n_tok ? tokens[g + lane] - r0 : -1;
            const bool near = k >= 0 && k < 8;
            if (__ballot(near) == 0ull) continue;
#pragma unroll
            for (int q = 0; q < 8; ++q) named |= __ballot(near && k == q) != 0ull ? 1u << q : 0u;
        }
        for (int64_t r = r0; r < min(r0 + 8, (int64_t)vocab); ++r) {
            if ((named >> (r - r0)) & 1u) continue;
            for (int32_t c = lane * 4; c < d; c += 256)
                *reinterpret_cast<f32x4_t *>(dtable + r * d + c) = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        return;
    }
    const int32_t strips = (d + 511) / 512;
    const int32_t t0 = (int32_t)quotient(wave, strips), col = (int32_t)(wave - (int64_t)t0 * strips) * 512 + lane * 8;
    if (t0 >= n_tok) return;
    const int32_t id = tokens[t0];
    if (id < 0 || id >= vocab) return;
    for (int32_t g = 0; g < t0; g += 64)
        if (__ballot(g + lane < t0 && tokens[g + lane] == id) != 0ull) return;  // the first one's wave does it
    const bool in = col < d;
    F8 acc = {};
    for (int32_t g = t0 / 64 * 64; g < n_tok; g += 64) {
        uint64_t left = __ballot(g + lane >= t0 && g + lane < n_tok && tokens[min(g + lane, n_tok - 1)] == id);
        while (left) {
            Raw8<T> x[U][BR];
            int n = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (left == 0ull) break;
                const int32_t t = g + __builtin_ctzll(left);
                left &= left - 1ull;
                ++n;
#pragma unroll
                for (int m = 0; m < BR; ++m) {
                    x[u][m] = Raw8<T>{};
                    if (in) x[u][m] = load_raw8(dh + ((int64_t)m * n_tok + t) * d + col);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u >= n) break;
#pragma unroll
                for (int m = 0; m < BR; ++m) {
                    const F8 v = x[u][m].get();
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc.v[i] += v.v[i];
                }
            }
        }
    }
    if (in) put_row(dtable + (int64_t)id * d + col, acc, scale, accumulate);
}

// Sorted positions per wave: 32, or 8 where that leaves the chip short of waves
// (a whole gradient of 1000 tokens x 256 channels: 14 us instead of 20, of 2048
// x 1024 over 32000 rows 28 instead of 34).
constexpr int64_t kLongItems = 65536;  // tokens times strips of 512 channels
int32_t run_chunk(int64_t n_tok, int32_t d) { return n_tok * ((d + 511) / 512) >= kLongItems ? 32 : 8; }
constexpr int kZeroRows = 8;   // table rows per wave of the zero part

// One wave per (run_chunk sorted positions, 512 channels) adds the chunk's rows
// in order.  A run that lies inside the chunk goes to its table row; the part
// of one that began earlier goes to lead[c], the part of one that began here
// and goes on to tail[c].  Blocks from sum_blocks on write zeros to the rows
// from zero_row on that have no tokens.
template <typename T, int BR>
__global__ __launch_bounds__(256) void embed_rows_kernel(const uint32_t *order, const int32_t *sid,
                                                         const uint32_t *start, int64_t n_tok, int32_t vocab,
                                                         int32_t d, const T *dh, float scale, bool accumulate,
                                                         float *dtable, float *lead, float *tail,
                                                         uint32_t sum_blocks, int64_t zero_row, int32_t chunk) {
    constexpr int U = sizeof(T) == 2 ? (BR == 1 ? 16 : 8) : (BR <= 2 ? 8 : 4);  // tokens whose rows are in flight
    const int lane = threadIdx.x & 63;
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (blockIdx.x >= sum_blocks) {
        const int64_t r0 = zero_row + (wave - (int64_t)sum_blocks * 4) * kZeroRows;
        for (int64_t r = r0; r < min(r0 + kZeroRows, (int64_t)vocab); ++r) {
            if (start[r] != start[r + 1]) continue;
            for (int32_t c = lane * 4; c < d; c += 256)
                *reinterpret_cast<f32x4_t *>(dtable + r * d + c) = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
        return;
    }
    const int32_t strips = (d + 511) / 512;
    const int64_t c = quotient(wave, strips);
    const int32_t col = (int32_t)(wave - c * strips) * 512 + lane * 8;
    const bool in = col < d;
    const int64_t n = start[vocab], base = c * chunk;
    if (base >= n) return;
    const int cnt = (int)min((int64_t)chunk, n - base);
    uint32_t my_tok = 0u;
    int32_t my_id = -1;
    if (lane < cnt) {
        my_tok = order[base + lane];
        my_id = sid[base + lane];
    }
    const int32_t before = base > 0 ? sid[base - 1] : -1;
    const int32_t after = base + cnt < n ? sid[base + cnt] : -1;
    bool started = __builtin_amdgcn_readlane(my_id, 0) != before;
    F8 acc = {};
    for (int k0 = 0; k0 < cnt; k0 += U) {
        Raw8<T> x[U][BR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t t = (uint32_t)__builtin_amdgcn_readlane((int)my_tok, min(k0 + u, cnt - 1));
#pragma unroll
            for (int m = 0; m < BR; ++m) {
                x[u][m] = Raw8<T>{};
                if (in) x[u][m] = load_raw8(dh + ((int64_t)m * n_tok + t) * d + col);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = k0 + u;
            if (k >= cnt) break;
#pragma unroll
            for (int m = 0; m < BR; ++m) {
                const F8 v = x[u][m].get();
#pragma unroll
                for (int i = 0; i < 8; ++i) acc.v[i] += v.v[i];
            }
            const int32_t id = __builtin_amdgcn_readlane(my_id, k);
            const int32_t next = k == cnt - 1 ? after : __builtin_amdgcn_readlane(my_id, min(k + 1, 63));
            const bool ends = next != id;
            if (!ends && k < cnt - 1) continue;
            if (in) {
                if (!started)
                    store8(lead + c * d + col, acc);
                else if (ends)
                    put_row(dtable + (int64_t)id * d + col, acc, scale, accumulate);
                else
                    store8(tail + c * d + col, acc);
            }
            acc = F8{};
            started = true;
        }
    }
}

// One workgroup per chunk and 256 channels: where a run starts in the chunk and
// goes on, its tail part plus the lead parts of the chunks behind it, a
// quarter of them each of the four waves, joined in order (a token that is a
// tenth of 32,768 leaves a hundred parts).
__global__ __launch_bounds__(256) void embed_join_kernel(const int32_t *sid, const uint32_t *start, int32_t vocab,
                                                         int32_t d, const float *lead, const float *tail,
                                                         float scale, bool accumulate, float *dtable, int32_t chunk) {
    __shared__ f32x4_t part[3][64];
    const int64_t c = blockIdx.x, base = c * chunk, n = start[vocab];
    if (base + chunk >= n) return;
    const int32_t id = sid[base + chunk - 1];
    const int64_t first = start[id], end = (int64_t)start[id + 1];
    if (first < base || end <= base + chunk) return;
    const int64_t k0 = c + 1, k1 = (end - 1) / chunk + 1;  // the chunks with a lead part
    const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t quarter = (k1 - k0 + 3) / 4, b = min(k0 + (w + 1) * quarter, k1);
    int64_t k = min(k0 + w * quarter, k1);
    const int32_t col = (int32_t)blockIdx.y * 256 + lane * 4;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    if (col < d) {
        if (w == 0) acc = *reinterpret_cast<const f32x4_t *>(tail + c * d + col);
        for (; k + 8 <= b; k += 8) {
            f32x4_t x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = *reinterpret_cast<const f32x4_t *>(lead + (k + u) * d + col);
#pragma unroll
            for (int u = 0; u < 8; ++u) acc += x[u];
        }
        for (; k < b; ++k) acc += *reinterpret_cast<const f32x4_t *>(lead + k * d + col);
    }
    if (w > 0) part[w - 1][lane] = acc;
    __syncthreads();
    if (w > 0 || col >= d) return;
    f32x4_t *dst = reinterpret_cast<f32x4_t *>(dtable + (int64_t)id * d + col);
    acc = (((acc + part[0][lane]) + part[1][lane]) + part[2][lane]) * scale;
    if (accumulate) acc += *dst;
    *dst = acc;
}

int64_t sort_blocks(int32_t vocab) { return ((int64_t)vocab + kBucket - 1) / kBucket; }
// Pieces of the tokens: of about kPiece, and at most a workgroup for each CU in
// all (the sort of 30,083 tokens over 1950 ids: 12.6 us against 33 in one piece,
// of 524,288 over 32,000: 193 against 464; pieces of 4096 13.9 us, of 8192 16.1;
// two workgroups a CU 229 us at the longest, four 346).  A vocabulary above
// 65,536 has more than 128 buckets, which leaves one piece.
constexpr int64_t kPiece = 2048;
int64_t sort_parts(int64_t n_tok, int32_t vocab) {
    return std::max<int64_t>(1, std::min((n_tok + kPiece - 1) / kPiece, 256 / sort_blocks(vocab)));
}
// Rows of the table that are filled beside the sort (at least one: d is far below kFillBeside).
int64_t fill_rows(int32_t vocab, int32_t d) {
    return std::min<int64_t>(vocab, std::max<int64_t>(1, kFillBeside / ((int64_t)d * 4)));
}

template <typename T>
void embed_few(const EmbedBwdArgs &a, hipStream_t s) {
    const uint32_t sum_blocks = (uint32_t)((a.n_tok * ((a.d + 511) / 512) + 3) / 4);
    const dim3 grid(sum_blocks + (a.accumulate ? 0u : (uint32_t)(((int64_t)a.vocab + 31) / 32)));
#define ENGRAM_EMBED_FEW(BR)                                                                                      \
    launch_kernel((embed_few_kernel<T, BR>), grid, dim3(256), s, a.tokens, (int32_t)a.n_tok, a.vocab, a.d,        \
                  static_cast<const T *>(a.dh), a.scale, a.accumulate, a.dtable, sum_blocks)
    switch (a.n_branches) {
        case 1: ENGRAM_EMBED_FEW(1); break;
        case 2: ENGRAM_EMBED_FEW(2); break;
        case 3: ENGRAM_EMBED_FEW(3); break;
        default: ENGRAM_EMBED_FEW(4); break;
    }
#undef ENGRAM_EMBED_FEW
}

template <typename T>
void embed_rows(const EmbedBwdArgs &a, hipStream_t s) {
    const int64_t chunks = embed_chunks(a.n_tok, a.d), strips = (a.d + 511) / 512;
    const uint32_t sum_blocks = (uint32_t)((chunks * strips + 3) / 4);
    const int64_t zero_row = a.accumulate ? a.vocab : fill_rows(a.vocab, a.d);
    const dim3 grid(sum_blocks + (unsigned)((a.vocab - zero_row + 4 * kZeroRows - 1) / (4 * kZeroRows)));
#define ENGRAM_EMBED_ROWS(BR)                                                                                   \
    launch_kernel((embed_rows_kernel<T, BR>), grid, dim3(256), s, a.order, a.sid, a.start, a.n_tok, a.vocab,    \
                  a.d, static_cast<const T *>(a.dh), a.scale, a.accumulate, a.dtable, a.lead, a.tail, sum_blocks, zero_row, run_chunk(a.n_tok, a.d))
    switch (a.n_branches) {
        case 1: ENGRAM_EMBED_ROWS(1); break;
        case 2: ENGRAM_EMBED_ROWS(2); break;
        case 3: ENGRAM_EMBED_ROWS(3); break;
        default: ENGRAM_EMBED_ROWS(4); break;
    }
#undef ENGRAM_EMBED_ROWS
}

}  // namespace

void launch_embed(engram_dtype dt, const int32_t *tokens, int64_t n_tok, int32_t vocab, const void *table, int32_t d,
                  int32_t n_branches, float scale, void *h, uint32_t *bad, hipStream_t s) {
    const int64_t items = n_tok * ((d + 511) / 512);
    const dim3 grid((unsigned)std::min<int64_t>((items + 3) / 4, (int64_t)1 << 22));
    if (dt == ENGRAM_BF16)
        launch_kernel(embed_kernel<uint16_t>, grid, dim3(256), s, tokens, n_tok, vocab,
                      static_cast<const uint16_t *>(table), d, n_branches, scale, static_cast<uint16_t *>(h), bad);
    else
        launch_kernel(embed_kernel<float>, grid, dim3(256), s, tokens, n_tok, vocab,
                      static_cast<const float *>(table), d, n_branches, scale, static_cast<float *>(h), bad);
}

int64_t embed_chunks(int64_t n_tok, int32_t d) {
    const int64_t c = run_chunk(n_tok, d);
    return (n_tok + c - 1) / c;
}

int64_t embed_short_tokens(int32_t d) { return (kLongItems - 1) / ((d + 511) / 512); }

bool embed_bwd_fits(int64_t n_tok, int32_t vocab, int32_t d) {
    // a launch holds fewer than 2^32 threads along x, and 65535 blocks along y
    const int64_t strips = (d + 511) / 512;
    const int64_t sums = std::max((embed_chunks(n_tok, d) * strips + 3) / 4, (std::min<int64_t>(n_tok, kFew) * strips + 3) / 4);
    return sums + ((int64_t)vocab + 31) / 32 < ((int64_t)1 << 24) &&
           embed_chunks(n_tok, d) < ((int64_t)1 << 24) && sort_blocks(vocab) < ((int64_t)1 << 21) &&
           (d + 255) / 256 <= 65535;
}

void launch_embed_bwd(engram_dtype dt, const EmbedBwdArgs &a, hipStream_t s) {
    if (a.n_tok <= kFew) {
        if (dt == ENGRAM_BF16)
            embed_few<uint16_t>(a, s);
        else
            embed_few<float>(a, s);
        return;
    }
    const int64_t fill = a.accumulate ? 0 : fill_rows(a.vocab, a.d) * a.d * 4;
    const int64_t parts = sort_parts(a.n_tok, a.vocab), sorts = sort_blocks(a.vocab) * parts, fills = (fill + kFillBytes - 1) / kFillBytes;
    launch_kernel(embed_sort_kernel, dim3((unsigned)(sorts + fills)), dim3(64 * kSortWaves), s, a.tokens, a.n_tok, a.vocab,
                  a.order, a.sid, a.start, (uint32_t)sorts, (int32_t)parts, a.dtable, fill);
    if (dt == ENGRAM_BF16)
        embed_rows<uint16_t>(a, s);
    else
        embed_rows<float>(a, s);
    const int64_t chunks = embed_chunks(a.n_tok, a.d);
    if (chunks > 1)
        launch_kernel(embed_join_kernel, dim3((unsigned)chunks, (unsigned)((a.d + 255) / 256)), dim3(256), s, a.sid,
                      a.start, a.vocab, a.d, a.lead, a.tail, a.scale, a.accumulate, a.dtable, run_chunk(a.n_tok, a.d));
}

}  // namespace engram
