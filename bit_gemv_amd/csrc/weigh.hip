// weigh.hip -- the attention weight that cached tokens receive, summed over a
// call's rows and the heads of a group (kv_cache_weigh).
//
// With codes c, scale s and zero z of a key and a row's log-sum-exp L,
//   weight_j += sum_i exp(scale s_j (q_i . c_j - z_j sum(q_i)) - L_i)
// Products are formed rows x keys: a lane then holds four rows of one key, sums
// them in its own register, and only the last sum crosses lanes. A key belongs
// to one block, which goes through all rows that see it, or to a few that share
// the rows and leave sums that a second launch adds up: no atomics, sums in a
// fixed order. Single tokens are bound by HBM: 64 sequences of up to 16384 tokens,
// 8 heads of 128, INT8, 156 us for 772 MB. Chunks are bound by the matrix and the
// vector units, whose times add up: of 64 scores of 128 elements a wave's products
// take 16 clocks, exponentials 8, scaling and sum 8. The last 500 rows of three
// prompts of up to 6000 tokens, 32 heads of 128, INT4: 68 us, 0.65 PFLOP/s.
#include "codes.hpp"
#include "kv.hpp"

#include <type_traits>

namespace lq {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 4;

// Steps of STEP keys of all sequences that have rows, one after another; a lane
// a sequence, 64 at a time, the first 64 kept.
struct Place {
    int64_t seq, start;  // start: the sequence's first step among all
    int steps;           // of the sequence
    KvRows rows;
};
template <int STEP>
struct Steps {
    struct Lane {
        KvRows rows;
        int64_t steps, upto;
    };
    const KvBatch &bt;
    const bool whole;
    const int shift, lane;
    Lane first;

    LQ_DEVICE Lane load(int64_t seq, int64_t before) const {
        Lane x{};
        if (seq < bt.b) {
            x.rows = kv_rows(bt, seq, shift, whole);
            x.steps = x.rows.n > 0 && x.rows.len > 0 ? (x.rows.len + STEP - 1) / STEP : 0;
        }
        x.upto = before + scan64(x.steps);
        return x;
    }
    LQ_DEVICE Steps(const WeighArgs &a, int l) : bt(a.batch), whole(a.whole), shift(a.c.page_shift), lane(l) { first = load(l, 0); }
    LQ_DEVICE int64_t total() const {
        int64_t sum = readlane64(first.upto, 63);
        for (int64_t s0 = 64; s0 < bt.b; s0 += 64) sum = readlane64(load(s0 + lane, sum).upto, 63);
        return sum;
    }
    // the sequence that holds step pos (below the total)
    LQ_DEVICE Place at(int64_t pos) const {
        Lane x = first;
        for (int64_t s0 = 0;;) {
            const uint64_t past = __ballot(x.upto > pos);
            if (past) {
                const int src = __ffsll((unsigned long long)past) - 1;
                Place p;
                p.seq = s0 + src;
                p.steps = (int)readlane64(x.steps, src);
                p.start = readlane64(x.upto, src) - p.steps;
                p.rows = {readlane64(x.rows.begin, src), readlane64(x.rows.n, src), readlane64(x.rows.first, src),
                          readlane64(x.rows.len, src)};
                return p;
            }
            const int64_t before = readlane64(x.upto, 63);
            s0 += 64;
            if (s0 >= bt.b) return Place{0, pos, 1, KvRows{0, 0, 0, 0}};  // not reached: pos is below the total
            x = load(s0 + lane, before);
        }
    }
};

// ---- few rows: keys streamed past one tile of 16 rows ----
//
// Wave w of a block walks its span's 32-key tiles w, w + 4, ..., the next two
// tiles' codes on their way: a tile's registers take the one after the next as
// soon as it has been multiplied. Two tiles on their way and one: 158 and 173 us
// for 64 sequences of up to 16384 tokens. Streaming loads and ordinary ones: there 157
// and 154, 64 up to 1000 18.0 and 17.2, 32 up to 8000 of 256-wide heads 91.3 and 88.7;
// but of 128-wide 38.3 and 39.6, INT4 26.5 and 28.3, 64-wide 22.8 and 25.8. Streaming
// is taken: it loses 5 % at most, ordinary loads up to 13.
template <int D, int BITS>
struct Few {
    static constexpr int kRow = D * BITS / 8;    // code bytes of a key
    static constexpr int KW = D * BITS / 128;    // code words per lane of 16 keys
    static constexpr int VEC = KW < 4 ? KW : 4;  // words per load
    static constexpr int NV = KW / VEC;
    static constexpr int CPV = VEC * 32 / BITS;  // codes per load
    static constexpr int STEPS = D / 32;         // MFMAs per 16 keys
    static constexpr float kMid = (float)(1 << (BITS - 1));
    struct Tile {
        uint32_t k[2][KW];
        float sk[2], zk[2], w;
    };
};
constexpr int kFewStep = 32 * kWaves;
constexpr int kLate = 64, kEarly = 4;  // tiles a wave holds the sums of, and up to which it holds none

template <int D, int BITS, bool SYM>
__global__ __launch_bounds__(64 * kWaves, 3) void weigh_few_kernel(WeighArgs a, int cap) {
    using C = Few<D, BITS>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int h = blockIdx.x % a.c.heads;
    const int block = blockIdx.x / a.c.heads;
    const int group = a.q_heads / a.c.heads;
    const int shift = a.c.page_shift, ps_mask = (1 << shift) - 1;
    const int pages = (int)a.c.pages;
    const uint32_t k_off = n * C::kRow + g * (C::VEC * 4);
    const uint32_t magic = fp16_magic();
    // weights of a wave's tiles, and the slots of their two groups of 16 keys
    __shared__ float held[kWaves][kLate * 32];
    __shared__ int64_t held_at[kWaves][kLate * 2];

    const Steps<kFewStep> sched(a, lane);
    const int64_t all = sched.total(), share = uniform_div(all + cap - 1, cap);
    const int64_t begin = block * share, end = begin + share < all ? begin + share : all;
    for (int64_t pos = begin; pos < end;) {
        const Place place = sched.at(pos);
        const KvRows &rows = place.rows;
        const int step0 = (int)(pos - place.start);
        const int step1 = end - place.start < place.steps ? (int)(end - place.start) : place.steps;
        pos = place.start + step1;
        const int32_t *const table = a.batch.table + place.seq * a.batch.max_pages;
        const uint32_t total = (uint32_t)rows.n * (uint32_t)group;
        const int kbeg = step0 * kFewStep;
        const int kstop = (int64_t)step1 * kFewStep < rows.len ? step1 * kFewStep : (int)rows.len;
        const int top = (kstop - 1) & ~15;
        const int first_key = kbeg + 32 * wave;
        const int its = kstop > first_key ? (kstop - first_key + kFewStep - 1) / kFewStep : 0;

        // pages of this lane's iteration of the wave, 64 iterations at a time
        int pid0 = 0, pid1 = 0;
        auto load_pages = [&](int it) {
            int k0 = first_key + kFewStep * (it + lane), k1 = k0 + 16;
            k0 = k0 < top ? k0 : top;
            k1 = k1 < top ? k1 : top;
            pid0 = table[k0 >> shift];
            pid1 = table[k1 >> shift];
            asm volatile("" : "+v"(pid0), "+v"(pid1));  // waited for here, not behind later loads
        };
        // Stores among the loads cost HBM more than their bytes (64 sequences, 21 MB
        // of weights beside 700 MB of keys: 169 us; 158 with the weights held in LDS
        // and written at the end of a run, 135 without any). Short runs, whose time
        // is latency, write each tile's.
        const bool late = its > kEarly;
        // One tile of 16 rows, as the launch's rule expects; more of them go
        // over the keys again and add to what the one before has written.
        for (uint32_t tile = 0; tile * 16 < total; ++tile) {
            const float *const before = tile ? a.out : a.weights;
            if (tile) {  // other lanes of the wave wrote some of it
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            }
            struct At {
                int64_t slot0, slot1;  // of the tile's two groups of 16 keys
                int key0, key1;        // their first keys; past any key for a page outside the pool
            };
            auto load = [&](typename C::Tile &x, int it) {
                At at;
                if (it > 0 && (it & 63) == 0) load_pages(it);
                const int key0 = first_key + kFewStep * it;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    int page = __builtin_amdgcn_readlane(u ? pid1 : pid0, it & 63);
                    const int key = key0 + 16 * u;
                    const bool in = (uint32_t)page < (uint32_t)pages;
                    (u ? at.key1 : at.key0) = in ? key : 0x7FFFFF00;
                    page = in ? page : 0;
                    const int kc = key < top ? key : top;
                    const int64_t slot = (((int64_t)page * a.c.heads + h) << shift) + (kc & ps_mask);
                    (u ? at.slot1 : at.slot0) = slot;
                    const uint8_t *kp = a.c.k_codes + slot * C::kRow;
#pragma unroll
                    for (int j = 0; j < C::NV; ++j) load_words<C::VEC, true>(x.k[u] + j * C::VEC, kp + j * 64 + k_off);
                    x.sk[u] = a.c.k_scales[slot + n];
                    if (!SYM) x.zk[u] = a.c.k_zeros[slot + n];
                }
                x.w = before ? before[(g & 1 ? at.slot1 : at.slot0) + n] : 0.0f;
                return at;
            };
            typename C::Tile xa, xb;  // two tiles of the wave are on their way at any time
            At ata{0, 0, 0, 0}, atb{0, 0, 0, 0};
            if (its > 0) {
                load_pages(0);
                ata = load(xa, 0);
            }
            if (its > 1) atb = load(xb, 1);
            // this lane's row as an operand; a row that has seen no key, or a NaN,
            // counts as zeros with a weight of nothing
            const uint32_t rr = tile * 16 + n;
            const bool live = rr < total;
            const uint32_t tok = live ? rr / (uint32_t)group : 0;
            const int qh = h * group + (int)(live ? rr - tok * (uint32_t)group : 0);
            const float lse = live ? a.lse[(rows.begin + tok) * a.q_heads + qh] : __builtin_inff();
            const bool ok = fabsf(lse) < __builtin_inff();
            f16x8 qf[C::STEPS];
            float c1, qsum = 0.0f;
            {
                u32x4 raw[C::STEPS];
                const uint16_t *qp = a.q + (rows.begin + tok) * a.q_stride + (int64_t)qh * D;
#pragma unroll
                for (int s = 0; s < C::STEPS; ++s) {
                    constexpr int SPV = C::CPV / 8;
                    const int d0 = C::CPV * (4 * (s / SPV) + g) + 8 * (s % SPV);
                    raw[s] = ok ? *reinterpret_cast<const u32x4 *>(qp + d0) : u32x4{0u, 0u, 0u, 0u};
                }
                c1 = q_to_fp16<C::STEPS, BITS, SYM, false>(raw, a.scale, qf, qsum);
                if (!SYM) qsum = add_halves16(add_halves32(qsum));
            }
            // rows 4 g + i of the products
            const float minus = ok ? -lse * kLog2e : -__builtin_inff();
            const int mine = live ? (int)(rows.first + tok) : -1;  // last position the row sees
            float c1r[4], nl[4], qs[4];
            int last[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c1r[i] = __shfl(c1, 4 * g + i);
                nl[i] = __shfl(minus, 4 * g + i);
                last[i] = __shfl(mine, 4 * g + i);
                if (!SYM) qs[i] = __shfl(qsum, 4 * g + i);
            }
            const int safe = (int)(rows.first + tile * 16 / (uint32_t)group);  // every row sees up to here

            auto step = [&](typename C::Tile &x, At &at, int it) {
                f32x4 t[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    t[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int s = 0; s < C::STEPS; ++s) {
                        f16x2 kf[4];
                        if constexpr (BITS == 8) {
                            int8_row(x.k[u][2 * s], kf);
                            int8_row(x.k[u][2 * s + 1], kf + 2);
                        } else {
                            const uint32_t w = x.k[u][s], w8 = w >> 8;
                            kf[0] = int4_low(w, magic); kf[1] = int4_high(w, magic);
                            kf[2] = int4_low(w8, magic); kf[3] = int4_high(w8, magic);
                        }
                        t[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(qf[s], join(kf), t[u], 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (!SYM) t[u][i] = __builtin_fmaf(C::kMid - x.zk[u], qs[i], t[u][i]);
                        t[u][i] *= x.sk[u];
                    }
                }
                const int k0 = at.key0 + n, k1 = at.key1 + n, key = g & 1 ? k1 : k0;
                const int64_t slot = (g & 1 ? at.slot1 : at.slot0) + n;
                const bool masked = at.key0 + 15 > safe || at.key1 + 15 > safe;
                const float was = key < rows.first || tile ? x.w : 0.0f;  // the call's own tokens start from nothing
                if (it + 2 < its) at = load(x, it + 2);
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float p = __builtin_amdgcn_exp2f(__builtin_fmaf(t[u][i], c1r[i], nl[i]));
                        if (masked) p = (u ? k1 : k0) > last[i] ? 0.0f : p;
                        sum[u] += p;
                    }
                sum[0] = add_halves32(add_halves16(sum[0]));
                sum[1] = add_halves32(add_halves16(sum[1]));
                const float mine = was + (g & 1 ? sum[1] : sum[0]);
                if (late) {
                    if (g < 2) held[wave][it % kLate * 32 + 16 * g + n] = mine;
                    if (g < 2 && n == 0) held_at[wave][it % kLate * 2 + g] = key < kstop ? slot : -1;
                } else if (g < 2 && key < kstop) {
                    a.out[slot] = mine;
                }
            };
            auto write = [&](int it0, int it1) {  // the held weights of tiles it0 to it1, two at a time
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll 4
                for (int i = it0; i < it1; i += 2) {
                    const int tile_of = i + (g >> 1), key = first_key + kFewStep * tile_of + 16 * (g & 1) + n;
                    const int64_t at16 = held_at[wave][tile_of % kLate * 2 + (g & 1)];
                    if (tile_of < it1 && key < kstop && at16 >= 0) a.out[at16 + n] = held[wave][i % kLate * 32 + lane];
                }
            };
            for (int it = 0; it < its; it += 2) {
                step(xa, ata, it);
                if (it + 1 < its) step(xb, atb, it + 1);
                if (late && (it + 2 >= its || (it + 2) % kLate == 0)) write(it - it % kLate, it + 2 < its ? it + 2 : its);
            }
        }
    }
}

// ---- many rows: keys in the waves' registers, rows streamed past them ----
//
// The codes less their zeros are integers of up to 9 bits, which bf16 holds
// exactly, so the rows are multiplied as they lie. Each wave turns the codes of
// TILES x 16 keys of its own into operands once and keeps them; the block brings
// the rows, 32 at a time, through two buffers in LDS. A lane's operands are one
// run of its key's bytes: of the products' D terms step s takes the 8-element
// chunks g S + s. Where a block for each run of keys would not fill the card,
// `splits` blocks share its rows, leave their sums in the workspace, and
// weigh_join_kernel adds them up.
template <int D, int BITS>
struct Many {
    static constexpr int TILES = D == 256 ? 2 : 4;
    static constexpr int KT = 16 * TILES * kWaves;    // keys of a block
    static constexpr int S = D / 32;                  // MFMAs per 16 keys
    static constexpr int RT = 2, ROWS = 16 * RT;      // row tiles and rows of a stage
    static constexpr int CHUNKS = D / 8;              // of 8 elements, a row
    static constexpr int LOADS = ROWS * CHUNKS / (64 * kWaves);  // chunks a thread and stage
    static constexpr int WORDS = S * BITS / 4;        // code words of a lane and key
    static constexpr float kMid = (float)(1 << (BITS - 1));
    struct Stage {
        u32x4 ops[RT][S][64];  // lane (n, g) in the place g 16 + (n ^ its chunk mod 16)
        float minus[ROWS];          // -lse in log2, -inf for a row that adds nothing
        int sees[ROWS];             // last position it sees
    };
    struct Load {
        u32x4 raw[LOADS];
        float lse[LOADS];
    };
};

// How the many-row kernel's work is shared out: `cap` blocks a key head walk the
// steps, the first `cut` of which `splits` blocks each share.
struct Shares {
    int64_t cap, cut;
    int splits;
    float *parts;  // [cut][splits][heads][keys of a step]
};

template <int D, int BITS, bool SYM>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 2 : 3) void weigh_many_kernel(WeighArgs a, Shares sh) {
    using C = Many<D, BITS>;
    constexpr int TILES = C::TILES;
    __shared__ typename C::Stage stage[2];
    __shared__ float rest[kWaves][16 * TILES];
    __shared__ int key_page[kWaves][16 * TILES];  // -1: not a key
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int h = blockIdx.x % a.c.heads;
    const uint32_t group = (uint32_t)a.q_heads / (uint32_t)a.c.heads;
    const int shift = a.c.page_shift, ps_mask = (1 << shift) - 1;
    const int pages = (int)a.c.pages;
    // the chunks this thread brings of a stage: one of its row, of every few rows
    constexpr int kStep = 64 * kWaves / C::CHUNKS;
    const int my_row = threadIdx.x / C::CHUNKS, my_chunk = threadIdx.x % C::CHUNKS;
    const uint32_t dtok = C::ROWS / group, drem = C::ROWS % group;
    const int64_t dq = dtok * a.q_stride + drem * D;
    const int dl = (int)(dtok * a.q_heads + drem);

    const Steps<C::KT> sched(a, lane);
    const int64_t all = sched.total();
    // items: the cut steps' splits, then whole steps
    const int64_t cut = all < sh.cut ? all : sh.cut, items = cut * sh.splits + (all - cut);
    for (int64_t item = blockIdx.x / a.c.heads; item < items; item += sh.cap) {
        const bool split = item < cut * sh.splits;
        const int64_t pos = split ? item / sh.splits : item - cut * (sh.splits - 1);
        const Place place = sched.at(pos);
        const KvRows &rows = place.rows;
        const int32_t *const table = a.batch.table + place.seq * a.batch.max_pages;
        const int k0 = (int)(pos - place.start) * C::KT;
        const uint32_t total = (uint32_t)rows.n * group;
        // rows before the first key see none of them
        const int64_t late = k0 - rows.first;
        uint32_t row0 = late <= 0 ? 0 : late < rows.n ? (uint32_t)late * group : total;
        int stages = (int)((total - row0 + C::ROWS - 1) / C::ROWS);
        if (split) {
            const int64_t share = item - pos * sh.splits;
            const int from = (int)(share * stages / sh.splits), to = (int)((share + 1) * stages / sh.splits);
            row0 += (uint32_t)from * C::ROWS;
            stages = to - from;
        }

        // This thread's rows go on by ROWS from stage to stage: dtok tokens and drem
        // heads, or a token more and the group's heads fewer.
        const uint16_t *const q0 = a.q + rows.begin * a.q_stride + (int64_t)h * group * D;
        const float *const lse0 = a.lse + rows.begin * a.q_heads + (int64_t)h * group;
        const uint16_t *qp[C::LOADS];
        const float *lp[C::LOADS];
        uint32_t rem[C::LOADS];
        int sees[C::LOADS];
#pragma unroll
        for (int i = 0; i < C::LOADS; ++i) {
            const uint32_t rr = row0 + my_row + i * kStep, tok = rr / group;
            rem[i] = rr - tok * group;
            sees[i] = (int)(rows.first + tok);
            qp[i] = q0 + tok * a.q_stride + rem[i] * D + 8 * my_chunk;
            lp[i] = lse0 + (int64_t)tok * a.q_heads + rem[i];
        }
        auto load = [&](typename C::Load &x, int st) {
            if (total - row0 >= (uint32_t)(st + 1) * C::ROWS) {
#pragma unroll
                for (int i = 0; i < C::LOADS; ++i) {
                    x.lse[i] = *lp[i];
                    x.raw[i] = *reinterpret_cast<const u32x4 *>(qp[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < C::LOADS; ++i) {
                    const bool live = row0 + (uint32_t)st * C::ROWS + my_row + i * kStep < total;
                    x.lse[i] = live ? *lp[i] : __builtin_inff();
                    x.raw[i] = live ? *reinterpret_cast<const u32x4 *>(qp[i]) : u32x4{0u, 0u, 0u, 0u};
                }
            }
        };
        auto store = [&](typename C::Load &x, typename C::Stage &to) {
            bool ok[C::LOADS], all_ok = true;
#pragma unroll
            for (int i = 0; i < C::LOADS; ++i) {
                ok[i] = fabsf(x.lse[i]) < __builtin_inff();
                all_ok &= ok[i];
            }
            // a row that has seen no key, or a NaN, counts as zeros with a weight of nothing
            if (!__all(all_ok)) {
#pragma unroll
                for (int i = 0; i < C::LOADS; ++i) {
                    x.raw[i] = ok[i] ? x.raw[i] : u32x4{0u, 0u, 0u, 0u};
                    x.lse[i] = ok[i] ? x.lse[i] : __builtin_inff();
                }
            }
#pragma unroll
            for (int i = 0; i < C::LOADS; ++i) {
                const int row = my_row + i * kStep;
                to.ops[row / 16][my_chunk % C::S][my_chunk / C::S * 16 + ((row ^ my_chunk) & 15)] = x.raw[i];
            }
            if (my_chunk == 0) {
#pragma unroll
                for (int i = 0; i < C::LOADS; ++i) {
                    to.minus[my_row + i * kStep] = -x.lse[i] * kLog2e;
                    to.sees[my_row + i * kStep] = sees[i];
                }
            }
#pragma unroll
            for (int i = 0; i < C::LOADS; ++i) {
                qp[i] += dq;
                lp[i] += dl;
                sees[i] += (int)dtok;
            }
            if (drem) {
#pragma unroll
                for (int i = 0; i < C::LOADS; ++i) {
                    rem[i] += drem;
                    if (rem[i] >= group) {
                        rem[i] -= group;
                        qp[i] += a.q_stride - (int64_t)group * D;
                        lp[i] += a.q_heads - (int)group;
                        ++sees[i];
                    }
                }
            }
        };
        typename C::Load x;
        if (stages > 0) load(x, 0);

        // the wave's keys: key 16 k + n of its own in lanes n
        const int kw = k0 + 16 * TILES * wave;
        int page[TILES];
        float scale[TILES], zero[TILES], acc[TILES];
        uint32_t w[TILES][C::WORDS];
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
            const int key = kw + 16 * k + n, kc = key < rows.len ? key : (int)rows.len - 1;
            page[k] = table[kc >> shift];
        }
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
            const int key = kw + 16 * k + n, kc = key < rows.len ? key : (int)rows.len - 1;
            const bool in = key < rows.len && (uint32_t)page[k] < (uint32_t)pages;
            page[k] = in ? page[k] : -1;
            const int64_t slot = (((int64_t)(in ? page[k] : 0) * a.c.heads + h) << shift) + (kc & ps_mask);
            const uint32_t *src = reinterpret_cast<const uint32_t *>(a.c.k_codes) + (slot * 4 + g) * C::WORDS;
#pragma unroll
            for (int i = 0; i < C::WORDS; i += 4) {
                if constexpr (C::WORDS >= 4) {
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(src + i);
                    w[k][i] = v[0]; w[k][i + 1] = v[1]; w[k][i + 2] = v[2]; w[k][i + 3] = v[3];
                } else {
                    const u32x2 v = *reinterpret_cast<const u32x2 *>(src);
                    w[k][0] = v[0]; w[k][1] = v[1];
                }
            }
            scale[k] = a.c.k_scales[slot];
            if (!SYM) zero[k] = a.c.k_zeros[slot];
            acc[k] = 0.0f;
        }
        bf16x8 kf[TILES][C::S];
        bool any_wide = false;
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
            key_page[wave][16 * k + n] = page[k];
            scale[k] = page[k] >= 0 ? scale[k] * (a.scale * kLog2e) : 0.0f;
            float near = C::kMid;
            if constexpr (!SYM) {
                const float z = page[k] >= 0 ? zero[k] : 0.0f;
                near = fminf(fmaxf(rintf(z), 0.0f), 2.0f * C::kMid - 1.0f);
                const float left = z - near;
                any_wide |= left != 0.0f;
                rest[wave][16 * k + n] = left;
            }
#pragma unroll
            for (int s = 0; s < C::S; ++s) {
                // INT4: even elements are the low nibbles of the bytes, odd ones the
                // high (hidden from the compiler, which otherwise shifts every code
                // by itself instead of converting bytes)
                uint32_t lo = w[k][(BITS == 8 ? 2 * s : s) % C::WORDS], hi = w[k][(BITS == 8 ? 2 * s + 1 : s) % C::WORDS];
                if constexpr (BITS == 4) {
                    lo = lo & 0x0F0F0F0Fu;
                    hi = hi >> 4 & 0x0F0F0F0Fu;
                    asm volatile("" : "+v"(lo), "+v"(hi));
                }
                u32x4 pairs;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t c0 = BITS == 8 ? (e < 2 ? lo : hi) >> 16 * (e % 2) : lo >> 8 * e;
                    const uint32_t c1 = BITS == 8 ? (e < 2 ? lo : hi) >> (16 * (e % 2) + 8) : hi >> 8 * e;
                    const bf16x2_t v{(__bf16)((float)(c0 & 255u) - near), (__bf16)((float)(c1 & 255u) - near)};
                    pairs[e] = __builtin_bit_cast(uint32_t, v);
                }
                kf[k][s] = __builtin_bit_cast(bf16x8, pairs);
            }
        }
        any_wide = !SYM && __any(any_wide);
        if (stages > 0) store(x, stage[0]);
        if (stages > 1) load(x, 1);
        __syncthreads();

        // rows from here on see all of the wave's keys
        const int64_t beyond = kw + 16 * TILES - 1 - rows.first;
        const uint32_t safe = beyond <= 0 ? 0 : beyond < rows.n ? (uint32_t)beyond * group : total;
        for (int st = 0; st < stages; ++st) {
            const typename C::Stage &b = stage[st & 1];
#pragma unroll
            for (int r = 0; r < C::RT; ++r) {
                bf16x8 qf[C::S];
#pragma unroll
                for (int s = 0; s < C::S; ++s)
                    qf[s] = __builtin_bit_cast(bf16x8, b.ops[r][s][g * 16 + ((n ^ (g * C::S + s)) & 15)]);
                const f32x4 nl = *reinterpret_cast<const f32x4 *>(&b.minus[16 * r + 4 * g]);
                // keys that some row of the tile does not see
                const bool masked = row0 + st * C::ROWS + 16 * r < safe;
                auto weigh = [&](auto masked_keys, auto wide_zeros) {
                    int last[4];
                    f32x4 qs{0.0f, 0.0f, 0.0f, 0.0f};  // the rows' sums
                    if constexpr (masked_keys) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) last[i] = b.sees[16 * r + 4 * g + i];
                    }
                    if constexpr (wide_zeros) {
                        bf16x8 ones;
#pragma unroll
                        for (int e = 0; e < 8; ++e) ones[e] = (__bf16)1.0f;
#pragma unroll
                        for (int s = 0; s < C::S; ++s) qs = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[s], ones, qs, 0, 0, 0);
                    }
#pragma unroll
                    for (int k = 0; k < TILES; ++k) {
                        f32x4 t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int s = 0; s < C::S; ++s) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[s], kf[k][s], t, 0, 0, 0);
                        if constexpr (wide_zeros) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) t[i] = __builtin_fmaf(-rest[wave][16 * k + n], qs[i], t[i]);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float p = __builtin_amdgcn_exp2f(__builtin_fmaf(t[i], scale[k], nl[i]));
                            if constexpr (masked_keys) p = kw + 16 * k + n > last[i] ? 0.0f : p;
                            acc[k] += p;
                        }
                    }
                };
                if (any_wide) weigh(std::true_type{}, std::true_type{});
                else if (masked) weigh(std::true_type{}, std::false_type{});
                else weigh(std::false_type{}, std::false_type{});
            }
            if (st + 1 < stages) store(x, stage[(st + 1) & 1]);
            if (st + 2 < stages) load(x, st + 2);
            lds_barrier();  // the next stage is written, and this one read by all
        }
#pragma unroll
        for (int k = 0; k < TILES; ++k) {
            const float sum = add_halves32(add_halves16(acc[k]));
            if (g != k % 4) continue;
            if (split) {
                sh.parts[(item * a.c.heads + h) * C::KT + 16 * (TILES * wave + k) + n] = sum;
            } else if (const int p = key_page[wave][16 * k + n]; p >= 0) {
                const int key = kw + 16 * k + n;
                const int64_t slot = (((int64_t)p * a.c.heads + h) << shift) + (key & ps_mask);
                // the call's own tokens start from nothing
                const bool old = a.weights && key < rows.first;
                a.out[slot] = (old ? a.weights[slot] : 0.0f) + sum;
            }
        }
    }
}

// Adds the splits' sums of the cut steps up, in order: a block a step and head,
// a thread a key.
template <int KT>
__global__ __launch_bounds__(KT) void weigh_join_kernel(WeighArgs a, Shares sh) {
    const int h = blockIdx.x % a.c.heads;
    const int64_t pos = blockIdx.x / a.c.heads;
    const int shift = a.c.page_shift;
    const Steps<KT> sched(a, threadIdx.x & 63);
    if (pos >= sched.total()) return;
    const Place place = sched.at(pos);
    const int64_t key = (pos - place.start) * KT + threadIdx.x;
    if (key >= place.rows.len) return;
    const int64_t page = kv_page(a.batch, place.seq, key, shift, a.c.pages);
    if (page < 0) return;
    const int64_t slot = ((page * a.c.heads + h) << shift) + (key & ((1 << shift) - 1));
    float sum = 0.0f;
#pragma unroll 4
    for (int i = 0; i < sh.splits; ++i) sum += sh.parts[((pos * sh.splits + i) * a.c.heads + h) * KT + threadIdx.x];
    const bool old = a.weights && key < place.rows.first;
    a.out[slot] = (old ? a.weights[slot] : 0.0f) + sum;
}

// The steps of KT keys that the bounds allow for and, where that many blocks do
// not fill the card, how many share each one's rows.
struct Cut {
    int64_t steps;
    int splits;
};
Cut cut_of(int64_t rows, int64_t group, int64_t heads, int64_t head_dim, int64_t b, int64_t room, int64_t max_rows,
           int64_t max_kv) {
    const int64_t n = max_rows <= 0 || max_rows > rows ? rows : max_rows, kv = max_kv <= 0 || max_kv > room ? room : max_kv;
    if (n * group <= 16) return {0, 1};
    const int64_t keys = head_dim == 256 ? Many<256, 8>::KT : Many<128, 8>::KT;
    const int64_t steps = b * ((kv + keys - 1) / keys < 1 ? 1 : (kv + keys - 1) / keys);
    // Two rounds of the three blocks a CU has room for, each of 128 rows or more.
    // One block for a run of keys and this: a prompt of 4096 tokens on 8 heads 1136
    // and 189 us, on one 1180 and 46; 4 x 500 rows over 3000 137 and 70; 64 rows over
    // 8000 25 and 27 (30 with 64 rows or more), 4 x 100 over 2000 on 2 heads 32 and 16.
    const int64_t fill = 1536 / (steps * heads), most = (n * group + 127) / 128;
    const int64_t splits = fill < most ? fill : most;
    return {splits > 1 ? steps : 0, splits > 1 ? (int)splits : 1};
}

}  // namespace

template <int D, int BITS, bool SYM>
static hipError_t launch(const WeighArgs &a, hipStream_t st) {
    const int64_t group = a.q_heads / a.c.heads, heads = a.c.heads, b = a.batch.b;
    const int64_t room = a.batch.max_pages << a.c.page_shift;
    const int64_t n = a.max_rows <= 0 || a.max_rows > a.batch.rows ? a.batch.rows : a.max_rows;
    const int64_t kv = a.max_kv <= 0 || a.max_kv > room ? room : a.max_kv;
    // blocks a key head: no more than `each` for each step of work, nor than `most` in all
    auto blocks = [&](int64_t step, int64_t each, int64_t most) {
        const int64_t steps = b * ((kv + step - 1) / step < 1 ? 1 : (kv + step - 1) / step) * each;
        const int64_t cap = (most + heads - 1) / heads;
        return cap < steps ? cap : steps;
    };
    if (n * group <= 16) {
        // Past one tile the keys would be read again: 64 sequences of 4 rows and 8
        // heads of a group over 4000 tokens 39 us here, 33 below; 16 of 3 rows over
        // 8000 39 and 32. 512, 768 and 1024 blocks, 64 sequences up to 16384: 166,
        // 165 and 178 us.
        const int cap = (int)blocks(kFewStep, 1, 768);
        hipLaunchKernelGGL((weigh_few_kernel<D, BITS, SYM>), dim3((uint32_t)(cap * heads)), dim3(64 * kWaves), 0, st, a, cap);
        return hipGetLastError();
    }
    constexpr int KT = Many<D, BITS>::KT;
    const Cut c = cut_of(a.batch.rows, group, heads, D, b, room, a.max_rows, a.max_kv);
    // more steps than that are walked: with no bound of the lengths most of a wide
    // table's steps may hold nothing
    const Shares sh{blocks(KT, c.splits, 1 << 12), c.steps, c.splits, static_cast<float *>(a.workspace)};
    hipLaunchKernelGGL((weigh_many_kernel<D, BITS, SYM>), dim3((uint32_t)(sh.cap * heads)), dim3(64 * kWaves), 0, st, a, sh);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || c.splits == 1) return e;
    hipLaunchKernelGGL(weigh_join_kernel<KT>, dim3((uint32_t)(c.steps * heads)), dim3(KT), 0, st, a, sh);
    return hipGetLastError();
}

int64_t weigh_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t b, int64_t max_pages,
                              int64_t page_size, int64_t max_rows, int64_t max_kv) {
    const Cut c = cut_of(rows, q_heads / heads, heads, head_dim, b, max_pages * page_size, max_rows, max_kv);
    const int64_t keys = head_dim == 256 ? Many<256, 8>::KT : Many<128, 8>::KT;
    return c.steps * c.splits * heads * keys * 4;
}

hipError_t launch_kv_weigh(const WeighArgs &a, hipStream_t st) {
#define LQ_WEIGH(D, BITS, SYM) \
    if (a.c.head_dim == D && a.c.bits == BITS && (a.c.symmetric != 0) == SYM) return launch<D, BITS, SYM>(a, st);
#define LQ_WEIGH_D(D) LQ_WEIGH(D, 4, false) LQ_WEIGH(D, 4, true) LQ_WEIGH(D, 8, false) LQ_WEIGH(D, 8, true)
    LQ_WEIGH_D(64) LQ_WEIGH_D(128) LQ_WEIGH_D(256)
#undef LQ_WEIGH_D
#undef LQ_WEIGH
    return hipErrorInvalidValue;
}

}  // namespace lq
