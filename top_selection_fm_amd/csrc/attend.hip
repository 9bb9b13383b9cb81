// attend.hip -- attention of query rows over a paged key/value cache: causal with a sliding
// window and first entries that stay visible (sinks), and the same for a tree of drafted tokens.
//
// Row r of a request and query head h (kv head h / G, G = n_heads / n_kv_heads):
//   x_s = scale q . k_s over the visible entries s,  o = sum_s softmax(x)_s v_s,  lse = ln sum e^x_s.
// The G heads of a kv head and a request's rows are flattened (row-major, heads inner) into the
// columns of one problem, so the entries are read once for 32 or more of them.
//
// A wave holds 32 columns.  Scores are formed transposed, S^T = K Q^T (entries x columns), on
// 32 x 32 MFMA tiles: lane j + 32 h then holds, for column j, the entries 8 (v / 4) + 4 h + v % 4
// of accumulator register v, so the softmax statistics of a column are per-lane values (the two
// halves of a column meet through one lane swap), and the exponentials are already where the
// second product O^T = V^T P^T wants its B operand, if the entries of a k step are taken in that
// order.  V^T's A operand comes from LDS through the transposing reads (ds_read_b64_tr_b16): no
// shuffle and no LDS round trip for P.  Statistics, sums and outputs are float32; for bf16 and
// fp8 caches the probabilities are rounded to bf16 for the second product (relative 2^-8 each,
// like the rounding of the output itself), their sum is taken before the rounding.
//
// The kernels:
//   attend_split_kernel  few columns (<= 32): the four waves of a workgroup hold the same columns
//                        and each streams tiles of its own, without barriers; bound by memory.
//   attend_block_kernel  more columns, bf16 and fp8: eight waves of 32 columns share each tile;
//                        bound by MFMA and the exponentials.
//   attend_tile_kernel   more columns, float32: four waves; bound by the float32 MFMAs.
// Each can split the entries over several workgroups; attend_merge_kernel joins the parts.
//
// Masks: each lane forms a word of visible entries for a tile; tiles every column sees whole skip
// the test.  A masked entry's key can hold anything (its score is replaced), and so can its
// value: 0 * inf would reach the sum through the product, so tiles with masked entries are
// searched for values that are not finite, and what those do is kept apart (Special, below).
#include <algorithm>
#include <type_traits>

#include "fm_internal.h"

namespace fm {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();
// A column's running maximum is raised only when a tile exceeds it by this many powers of two:
// until then the exponentials stay below 2^8, far from overflow, and the sums need no rescaling.
constexpr float kLazy = 8.f;

// The two halves' values of a column (of lane j and lane j + 32), in both lanes.
struct Halves {
    uint32_t lo, hi;
};
__device__ __forceinline__ Halves halves(uint32_t x) {
    const auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return {s[0], s[1]};
}
__device__ __forceinline__ float both_max(float x) {
    const Halves y = halves(__float_as_uint(x));
    return fmaxf(__uint_as_float(y.lo), __uint_as_float(y.hi));
}
__device__ __forceinline__ float both_sum(float x) {
    const Halves y = halves(__float_as_uint(x));
    return __uint_as_float(y.lo) + __uint_as_float(y.hi);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

__device__ __forceinline__ f32x16 mma_bf16(const u32x4 &a, const u32x4 &b, const f32x16 &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A per-lane value the compiler cannot carry from one tile to the next: what is derived from it (a
// dozen swizzled LDS addresses) is formed again for every tile, which costs less than holding it.
__device__ __forceinline__ uint32_t again(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}

// A value that is formed here, not where it is used.
__device__ __forceinline__ void here(float &x) { asm volatile("" : "+v"(x)); }

template <int N> __device__ __forceinline__ void wait_vm() {     // s_waitcnt vmcnt(N), others left alone
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// A tile in LDS: E entries (rows) of D values, bf16 (64 rows) or float32 (32 rows), in 16-byte
// pieces.  Row r's piece p sits at piece p ^ swz(r) of the row, so that the reads below touch
// every bank group evenly: 16 rows at one piece (scores, bf16 and float32), or 8 rows at two
// (transposing reads of bf16 values) or at eight (float32 values) neighbouring pieces.
template <int FMT, int D>
struct Tile {
    static constexpr bool F32 = FMT == KEY_F32;
    static constexpr int E = F32 ? 32 : 64;              // entries
    static constexpr int SUB = E / 32;                   // 32-entry MFMA tiles
    static constexpr int ROW = D * (F32 ? 4 : 2);        // bytes of a row
    static constexpr int NP = ROW / 16;                  // pieces of a row
    static constexpr int BYTES = E * ROW;
    static constexpr int DT = D / 32;                    // 32-value tiles of the output
    static constexpr int QR = F32 ? D / 8 : D / 16;      // 16-byte query registers of a lane

    __device__ static __forceinline__ int swz_k(int r) {
        if constexpr (F32) return (r & 3) | ((r & 4) << 1) | ((r & 8) >> 1);
        else if constexpr (NP == 16) return r & 15;
        else return (r >> 1) & 7;
    }
    __device__ static __forceinline__ int swz_v(int r) {
        if constexpr (F32) return swz_k(r);
        else if constexpr (NP == 16) return 2 * (r & 7);
        else return 2 * ((r >> 1) & 3);
    }
};

template <int FMT, int D> using QRegs = u32x4[Tile<FMT, D>::QR];
// Scores (then probabilities) of NS 32-entry tiles, and their packed form.
template <int NS> using SRegs = f32x16[NS];
template <int NS> using PRegs = u32x4[NS][2];

// One problem's columns: position, limits and masks of the lane's row.
struct Col {
    int pos;              // position of the row
    int lo, hi;           // entries [lo, hi) of the window, [0, sink) of the first ones
    int sink;
    bool valid;
    const uint64_t *mask; // tree: the row's bits (bit j: entry base + j), or null
    int base, n;
};

__device__ __forceinline__ uint64_t low_bits(int n) {     // bits 0 .. n - 1
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}
__device__ __forceinline__ uint64_t range_bits(int a, int b, int s0) {   // entries [a, b) of s0 ..
    return low_bits(b - s0) & ~low_bits(a - s0);
}

// The visible entries among s0 .. s0 + 63 of a column.
__device__ __forceinline__ uint64_t visible(const Col &c, int s0, int64_t mask_ld) {
    uint64_t w = range_bits(c.lo, c.hi, s0) | range_bits(0, c.sink, s0);
    if (c.mask && s0 + 63 >= c.base && s0 < c.base + c.n) {
        const int off = s0 - c.base;                      // bit of the tile's first entry
        uint64_t d;
        if (off < 0) {
            d = c.mask[0] << -off;                        // -off <= 63
        } else {
            const int i = off >> 6, sh = off & 63;        // off < n <= 64 mask_ld
            d = c.mask[i] >> sh;
            if (sh && i + 1 < mask_ld) d |= c.mask[i + 1] << (64 - sh);
        }
        w |= d & range_bits(c.base, c.base + c.n, s0);
    }
    return w;
}

// The lane's column R of request b (rows row0 .. row0 + n - 1, len entries).
__device__ __forceinline__ Col make_col(const AttendArgs &A, int R, int row0, int n, int len) {
    Col c;
    const int i = R / A.G;
    c.valid = i < n;
    c.n = n;
    c.base = len - n;
    c.pos = len - n + i;
    c.mask = nullptr;
    c.hi = c.pos + 1;
    if (A.tree_mask) {
        c.mask = A.tree_mask + (int64_t)(row0 + (c.valid ? i : 0)) * A.mask_ld;
        int seen = 0;
#pragma unroll 1
        for (int j = 0; j < n; j += 64) seen += __popcll(c.mask[j >> 6] & low_bits(n - j));
        c.pos = c.base + seen - 1;
        c.hi = c.base;
    }
    c.hi = max(c.hi, 0);
    c.lo = max(max(c.pos, 0) - (A.window - 1), 0);
    c.sink = min(A.n_sink, c.hi);
    if (c.lo >= c.hi) c.lo = c.hi;
    return c;
}

template <int E> __device__ __forceinline__ int tiles_of(int entries) {    // entries >= 0, up to 2^31 - 1
    return (int)(((unsigned)entries + E - 1) / E);
}
// Tiles of a workgroup's rows i0 .. i1: the first ones up to the sinks, then from the window on.
struct Span {
    int first;        // tiles 0 .. first - 1
    int from, count;  // then tiles from ..; count in all
    __device__ int at(int i) const { return i < first ? i : from + i - first; }
};
template <int E>
__device__ __forceinline__ Span make_span(const AttendArgs &A, int i0, int i1, int n, int len) {
    Span s{0, 0, 0};
    const int hi = A.tree_mask ? len : len - n + i1 + 1;
    if (i0 > i1 || hi <= 0) return s;
    // a row of a tree sits at base - 1 or later
    const int p0 = A.tree_mask ? len - n - 1 : len - n + i0;
    const int lo = max(max(p0, 0) - (A.window - 1), 0);
    s.first = tiles_of<E>(min(A.n_sink, hi));
    s.from = max(lo / E, s.first);
    s.count = s.first + max(tiles_of<E>(hi) - s.from, 0);
    return s;
}

template <int FMT, int D>
struct State {
    f32x16 o[Tile<FMT, D>::DT];
    float m, l;       // m: maximum in score units (both halves alike), l: the lane's own entries
    // what exponentials are taken against: m times c, or for float32 m (a difference first, so that an
    // exponent's error goes with its size and not the maximum's); 0 while nothing was seen
    float mc;
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int t = 0; t < Tile<FMT, D>::DT; ++t)
#pragma unroll
            for (int v = 0; v < 16; ++v) o[t][v] = 0.f;
        m = kNegInf;
        l = mc = 0.f;
    }
};

// The lane's queries: 16-byte pieces; rows past the problem read as zeros.
template <int FMT, int D>
__device__ __forceinline__ void load_q(QRegs<FMT, D> &q, const AttendArgs &A, int R, int row0,
                                       int hk, bool valid) {
    const int h = __lane_id() >> 5;
    const int64_t row = row0 + R / A.G;
    const int64_t at = row * A.q_ld + (int64_t)(hk * A.G + R % A.G) * D;
    const uint8_t *p = (const uint8_t *)A.q + at * (FMT == KEY_F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < Tile<FMT, D>::QR; ++i) {
        const u32x4 zero = {0u, 0u, 0u, 0u};
        q[i] = valid ? *(const u32x4 *)(p + 32 * i + 16 * h) : zero;
    }
}

// Byte offsets in a tile of the lane's first reads; the others differ by an exclusive or and by
// whole rows.
template <int FMT, int D>
__device__ __forceinline__ uint32_t key_lane() {
    using TL = Tile<FMT, D>;
    const int ln = __lane_id(), h = ln >> 5, r = ln & 31;
    return (uint32_t)(r * TL::ROW + 16 * (h ^ TL::swz_k(r)));
}
template <int FMT, int D>
__device__ __forceinline__ uint32_t value_lane() {
    using TL = Tile<FMT, D>;
    const int ln = __lane_id(), h = ln >> 5;
    if constexpr (TL::F32) {
        const int j = ln & 31, r = 4 * h;
        return (uint32_t)(r * TL::ROW + 16 * ((j >> 2) ^ TL::swz_v(r)) + 4 * (j & 3));
    } else {
        const int i = ln & 15, g = (ln >> 4) & 1, r = 4 * h + (i >> 2);
        return (uint32_t)(r * TL::ROW + 16 * ((2 * g + ((i & 3) >> 1)) ^ TL::swz_v(r)) + 8 * (i & 1));
    }
}

// S^T of one 32-entry tile; lane: key_lane.
template <int FMT, int D>
__device__ __forceinline__ f32x16 scores(const uint8_t *kt, uint32_t lane, int sub, const QRegs<FMT, D> &q) {
    using TL = Tile<FMT, D>;
    f32x16 s;
#pragma unroll
    for (int v = 0; v < 16; ++v) s[v] = 0.f;
    // eight reads go out before the first product waits for one: a wave may be alone on its SIMD
    constexpr int U = TL::QR < 8 ? TL::QR : 8;
#pragma unroll
    for (int i0 = 0; i0 < TL::QR; i0 += U) {
        u32x4 a[U];
#pragma unroll
        for (int i = 0; i < U; ++i) a[i] = *(const u32x4 *)(kt + 32 * sub * TL::ROW + (lane ^ (uint32_t)(32 * (i0 + i))));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if constexpr (TL::F32) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    s = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[i][c]), __uint_as_float(q[i0 + i][c]), s, 0, 0, 0);
            } else {
                s = mma_bf16(a[i], q[i0 + i], s);
            }
        }
    }
    return s;
}

// Column sums over the entries of NS 32-entry tiles: o[d, column] += sum_e f(V[e, d]) P[e, column],
// f applied to the operand registers; lane: value_lane.  The values of 32 dims are read while the
// ones before are weighed.
template <int FMT, int D, int NS, class F>
__device__ __forceinline__ void weigh(const uint8_t *vt, uint32_t lane, const SRegs<NS> &p, const PRegs<NS> &pk,
                                      f32x16 (&o)[D / 32], F f) {
    using TL = Tile<FMT, D>;
    constexpr int N = TL::F32 ? 16 : 8 * NS;              // operand dwords
    uint32_t x[2][N];
    auto read = [&](uint32_t (&x)[N], int t) {
        if constexpr (TL::F32) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int r = 8 * (v >> 2) + (v & 3);     // and 4 h, in lane
                x[v] = *(const uint32_t *)(vt + (lane ^ (uint32_t)(16 * TL::swz_v(r) ^ 128 * t)) + r * TL::ROW);
            }
        } else {
            const uint8_t *at = vt + (lane ^ (uint32_t)(64 * t));
#pragma unroll
            for (int i = 0; i < 4 * NS; ++i) {            // rows 8 i and on: one swizzle for all
                const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4 *)(at + 8 * i * TL::ROW)));
                x[2 * i] = a[0];
                x[2 * i + 1] = a[1];
            }
        }
    };
    read(x[0], 0);
#pragma unroll
    for (int t = 0; t < TL::DT; ++t) {
        if (t + 1 < TL::DT) read(x[(t + 1) & 1], t + 1);
        __builtin_amdgcn_sched_barrier(0);
        const uint32_t (&y)[N] = x[t & 1];
        if constexpr (TL::F32) {
#pragma unroll
            for (int v = 0; v < 16; ++v)
                o[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(f(y[v])), p[0][v], o[t], 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * NS; ++i) {
                const u32x4 a = {f(y[4 * i]), f(y[4 * i + 1]), f(y[4 * i + 2]), f(y[4 * i + 3])};
                o[t] = mma_bf16(a, pk[i / 2][i % 2], o[t]);
            }
        }
    }
}

template <int FMT, int NS>
__device__ __forceinline__ void pack_p(const SRegs<NS> &p, PRegs<NS> &pk) {
    if constexpr (FMT != KEY_F32) {
#pragma unroll
        for (int sub = 0; sub < NS; ++sub)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    pk[sub][ks][w] = pack_bf16(p[sub][8 * ks + 2 * w], p[sub][8 * ks + 2 * w + 1]);
    }
}

// Columns' sums that a visible value which is not finite has reached: bits (column, value) of
// 0 * inf or NaN, +inf and -inf, applied to the sums before they leave the wave.
template <int D>
struct Special {
    uint32_t any;
    uint32_t nan[32][D / 32], up[32][D / 32], down[32][D / 32];
    uint32_t vis[32][2], dead[32][2];     // scratch: the columns' visible entries, and those with p = 0
};
template <int D>
__device__ __forceinline__ void clear_special(Special<D> &sp) {
    uint32_t *x = &sp.any;
#pragma unroll 1
    for (int i = __lane_id(); i < (int)(sizeof(Special<D>) / 4); i += 64) x[i] = 0;
}

// Marks what the infinities and NaNs of NS 32-entry tiles (at vt) do to the columns that see them;
// vis: bit e for entry e.  Rolled loops over LDS: such tiles are rare, and the wave's registers
// stay where they are.
template <int FMT, int D, int NS>
__device__ __forceinline__ void mark_special(const uint8_t *vt, const SRegs<NS> &p, uint64_t vis, Special<D> &sp) {
    using TL = Tile<FMT, D>;
    const int ln = __lane_id(), h = ln >> 5;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        uint32_t own = 0;
#pragma unroll
        for (int v = 0; v < 16; ++v) own |= p[i][v] == 0.f ? 1u << (8 * (v >> 2) + (v & 3)) : 0u;
        own <<= 4 * h;
        const Halves y = halves(own);
        const uint32_t both = y.lo | y.hi;
        if (ln < 32) {
            sp.vis[ln][i] = (uint32_t)(vis >> (32 * i));
            sp.dead[ln][i] = both;
        }
    }
    if (ln == 0) sp.any = 1;
    __builtin_amdgcn_wave_barrier();
    constexpr int W = TL::F32 ? 1 : 2;                     // values of a dword
#pragma unroll 1
    for (int x = ln; x < NS * 32 * TL::ROW / 4; x += 64) {
        const int r = x / (TL::ROW / 4), at = x % (TL::ROW / 4);
        const int d0 = (4 * ((at >> 2) ^ TL::swz_v(r)) + (at & 3)) * W;
        const uint32_t word = *(const uint32_t *)(vt + 4 * x);
#pragma unroll 1
        for (int k = 0; k < W; ++k) {
            const uint32_t y = W == 1 ? word : k ? word & 0xffff0000u : word << 16;
            if ((y & 0x7f800000u) != 0x7f800000u) continue;
            const int d = d0 + k;
            const bool isnan = (y & 0x007fffffu) != 0;
#pragma unroll 1
            for (int c = 0; c < 32; ++c) {
                if (!((sp.vis[c][r >> 5] >> (r & 31)) & 1)) continue;
                const bool zero = (sp.dead[c][r >> 5] >> (r & 31)) & 1;
                uint32_t *to = isnan || zero ? sp.nan[c] : y >> 31 ? sp.down[c] : sp.up[c];
                atomicOr(&to[d >> 5], 1u << (d & 31));
            }
        }
    }
    __builtin_amdgcn_wave_barrier();
}

template <int FMT, int D>
__device__ __forceinline__ void apply_special(const Special<D> &sp, State<FMT, D> &st) {
    if (!sp.any) return;
    const int ln = __lane_id(), j = ln & 31, h = ln >> 5;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int bit = 8 * (v >> 2) + 4 * h + (v & 3);
            if ((sp.up[j][t] >> bit) & 1) st.o[t][v] += __builtin_inff();
            if ((sp.down[j][t] >> bit) & 1) st.o[t][v] -= __builtin_inff();
            if ((sp.nan[j][t] >> bit) & 1) st.o[t][v] = __builtin_nanf("");
        }
}

// A dword of values with those that are not finite taken as zeros.
template <bool F32>
__device__ __forceinline__ uint32_t finite_only(uint32_t x) {
    if constexpr (F32) return (x & 0x7f800000u) == 0x7f800000u ? 0u : x;
    const uint32_t lo = (x & 0x00007f80u) == 0x00007f80u ? 0u : 0x0000ffffu;
    const uint32_t hi = (x & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u;
    return x & (lo | hi);
}

// Whether any value of the tile is not finite (a wave-uniform answer).
template <int FMT, int D>
__device__ __forceinline__ bool any_special(const uint8_t *vt) {
    using TL = Tile<FMT, D>;
    uint32_t bad = 0;
#pragma unroll
    for (int i = 0; i < TL::BYTES / 1024; ++i) {
        const u32x4 x = *(const u32x4 *)(vt + 1024 * i + 16 * __lane_id());
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if constexpr (TL::F32) bad |= (x[w] & 0x7f800000u) + 0x00800000u;
            else bad |= ((x[w] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        }
    }
    return __ballot((bad & 0x80008000u) != 0) != 0;
}

// fp8: scores times their entries' key scales.
template <int NS>
__device__ __forceinline__ void scale_scores(SRegs<NS> &s, const float *ks) {
    const int h = __lane_id() >> 5;
#pragma unroll
    for (int sub = 0; sub < NS; ++sub)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const f32x4 k = *(const f32x4 *)(ks + 32 * sub + 8 * a + 4 * h);
#pragma unroll
            for (int b = 0; b < 4; ++b) s[sub][4 * a + b] *= k[b];
        }
}

// Scores of the entries whose bit in vis is clear become -inf.
template <int NS>
__device__ __forceinline__ void hide(SRegs<NS> &s, uint64_t vis) {
    const uint64_t w = vis >> (4 * (__lane_id() >> 5));
#pragma unroll
    for (int sub = 0; sub < NS; ++sub) {
        const uint32_t half = (uint32_t)(w >> (32 * sub));
#pragma unroll
        for (int v = 0; v < 16; ++v) s[sub][v] = half & (1u << (8 * (v >> 2) + (v & 3))) ? s[sub][v] : kNegInf;
    }
}

template <int NS>
__device__ __forceinline__ float max_of(const SRegs<NS> &s) {
    float mx = s[0][0];
#pragma unroll
    for (int sub = 0; sub < NS; ++sub)
#pragma unroll
        for (int v = 0; v < 16; ++v) mx = fmaxf(mx, s[sub][v]);
    return mx;
}

// The column's maximum, raised (and the sums with it) where mx, the lane's new scores', calls for it.
template <int FMT, int D>
__device__ __forceinline__ void raise_max(float mx, float c, State<FMT, D> &st) {
    mx = both_max(mx);
    // where nothing was seen yet, m is -inf and any score exceeds it by inf
    if (__builtin_amdgcn_ballot_w64((mx - st.m) * c > kLazy)) {
        const float m = fmaxf(st.m, mx);
        const float a = st.m == kNegInf ? 0.f : __builtin_amdgcn_exp2f((st.m - m) * c);
        st.m = m;
        st.mc = m == kNegInf ? 0.f : FMT == KEY_F32 ? m : m * c;
        st.l *= a;
#pragma unroll
        for (int t = 0; t < Tile<FMT, D>::DT; ++t)
#pragma unroll
            for (int v = 0; v < 16; ++v) st.o[t][v] *= a;
    }
}

// Scores to exponentials, their sum to l, and (fp8; vs: the entries' value scales) scaled for the
// product with the codes.  c: scale * log2 e.
template <int FMT, int D, int NS>
__device__ __forceinline__ void exponentials(SRegs<NS> &s, bool masked, float c, const float *vs, State<FMT, D> &st) {
    const int h = __lane_id() >> 5;
    float sum[2] = {st.l, 0.f};
#pragma unroll
    for (int sub = 0; sub < NS; ++sub)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            s[sub][v] = __builtin_amdgcn_exp2f(FMT == KEY_F32 ? (s[sub][v] - st.mc) * c : fmaf(s[sub][v], c, -st.mc));
            sum[v & 1] += s[sub][v];
        }
    st.l = sum[0] + sum[1];
    if constexpr (FMT == KEY_FP8) {
#pragma unroll
        for (int sub = 0; sub < NS; ++sub)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const f32x4 k = *(const f32x4 *)(vs + 32 * sub + 8 * a + 4 * h);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int v = 4 * a + b;
                    const float y = s[sub][v] * k[b];
                    s[sub][v] = masked && s[sub][v] == 0.f ? 0.f : y;   // a masked entry's scale may be anything
                }
            }
    }
}

template <int FMT, int D, int NS>
__device__ __forceinline__ void soften(SRegs<NS> &s, bool masked, uint64_t vis, float c, const float *ks, const float *vs,
                                       State<FMT, D> &st) {
    if constexpr (FMT == KEY_FP8) scale_scores<NS>(s, ks);
    if (masked) hide<NS>(s, vis);
    raise_max<FMT, D>(max_of<NS>(s), c, st);
    exponentials<FMT, D, NS>(s, masked, c, vs, st);
}

// The values of NS 32-entry tiles at vt; special: some are not finite and some entries are masked.
template <int FMT, int D, int NS>
__device__ __forceinline__ void add_values(const uint8_t *vt, uint32_t lane, const SRegs<NS> &p, bool special,
                                           uint64_t vis, State<FMT, D> &st, Special<D> &sp) {
    PRegs<NS> pk;
    pack_p<FMT, NS>(p, pk);
    if (special) {
        mark_special<FMT, D, NS>(vt, p, vis, sp);
        weigh<FMT, D, NS>(vt, lane, p, pk, st.o, [](uint32_t x) { return finite_only<FMT == KEY_F32>(x); });
        return;
    }
    weigh<FMT, D, NS>(vt, lane, p, pk, st.o, [](uint32_t x) { return x; });
}

// Copy of a tile from the pool straight into LDS: instruction n of the tile moves 64 pieces.  The
// lane's source offset within an instruction's 1 KB is one value but for an exclusive or with n's
// part of the swizzle.
template <int FMT, int D, bool KEYS>
__device__ __forceinline__ void copy_pieces(const uint8_t *src, uint8_t *dst, int n) {
    using TL = Tile<FMT, D>;
    constexpr int RI = 1024 / TL::ROW;                    // rows of an instruction
    const uint32_t ln = again(__lane_id()), r = ln / TL::NP, at = ln % TL::NP;
    auto swz = [](int r) { return KEYS ? TL::swz_k(r) : TL::swz_v(r); };
    const uint32_t lane = (uint32_t)(r * TL::ROW + 16 * (at ^ swz(r)));
    const uint32_t ofs = lane ^ (uint32_t)(16 * swz(RI * n));   // swz(RI n + r) = swz(RI n) ^ swz(r)
    __builtin_amdgcn_global_load_lds((const void *)(src + 1024 * n + ofs), (lds_void *)(dst + 1024 * n), 16, 0, 0);
}

constexpr auto as_is = [](int, int, u32x4 y, float) { return y; };   // a piece as it was loaded

// fp8 tiles pass through registers: 16 codes a piece, widened exactly to bf16.
template <int N>
struct CodeRegs {
    u32x4 x[N];
    float scale;
};
// N pieces a thread, NT threads; scales are loaded by the first 64 threads or (OWN, N = 1) by each
// for its piece.
template <int N, int NT, bool OWN = false>
__device__ __forceinline__ void load_codes(CodeRegs<N> &c, const uint8_t *src, uint32_t tid) {
    const uint32_t lane = (tid >> 3) * kRowFp8 + 16 * (tid & 7);
#pragma unroll
    for (int i = 0; i < N; ++i) c.x[i] = *(const u32x4_u *)(src + lane + (NT / 8) * kRowFp8 * i);
    if constexpr (OWN) c.scale = *(const float *)(src + (tid >> 3) * kRowFp8 + kDim);
    else if (tid < 64) c.scale = *(const float *)(src + tid * kRowFp8 + kDim);
}
template <int N, int NT, bool KEYS, bool OWN = false, class F>
__device__ __forceinline__ void put_codes(const CodeRegs<N> &c, uint8_t *dst, float *scales, uint32_t tid, F fix) {
    using TL = Tile<KEY_FP8, kDim>;
    auto swz = [](int r) { return KEYS ? TL::swz_k(r) : TL::swz_v(r); };
    const uint32_t r = tid >> 3, lane = r * TL::ROW + 16 * ((2 * (tid & 7)) ^ swz(r));
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            u32x4 y;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t d = c.x[i][2 * o + w];
                y[2 * w] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, false));
                y[2 * w + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, 1.0f, true));
            }
            *(u32x4 *)(dst + (lane ^ (uint32_t)(16 * (o ^ swz(NT / 8 * i)))) + NT / 8 * i * TL::ROW) =
                fix(r + NT / 8 * i, 2 * (tid & 7) + o, y, c.scale);
        }
    if constexpr (OWN) {
        if ((tid & 7) == 0) scales[r] = c.scale;
    } else {
        if (tid < 64) scales[tid] = c.scale;
    }
}

// The page of tile `t` of request b, or -1 where it is not mapped.
template <int FMT, int D>
__device__ __forceinline__ int page_of(const AttendArgs &A, int b, int t) {
    // the table is not written meanwhile: a scalar load, which no copy in flight has to be waited for
    typedef const int32_t __attribute__((address_space(4))) *table;
    const int page = ((table)(uintptr_t)A.bt)[(int64_t)b * A.bt_ld + (int64_t)t * Tile<FMT, D>::E / kPage];
    return page >= 0 && page < A.n_phys ? page : -1;
}
// Where that tile starts in a pool.
template <int FMT, int D>
__device__ __forceinline__ int64_t tile_at(const AttendArgs &A, int page, int hk, int t) {
    constexpr int row = FMT == KEY_FP8 ? kRowFp8 : Tile<FMT, D>::ROW;
    return (((int64_t)page * A.n_kv + hk) * kPage + (int64_t)t * Tile<FMT, D>::E % kPage) * row;
}

// A problem's request, rows and length; the host's bounds hold whatever the device arrays say.
struct Req {
    int row0, n, len;
};
__device__ __forceinline__ Req request(const AttendArgs &A, int b) {
    Req r;
    r.row0 = max(0, min(A.q_start[b], A.T));
    r.n = max(0, min(min(A.q_start[b + 1], A.T) - r.row0, A.max_rows));
    r.len = max(0, min(A.seq_lens[b], A.max_len));
    return r;
}

// Column outputs.  stage: D floats of each of 32 columns, row c's 16-byte piece p at p ^ (c & 15).
template <int D>
__device__ __forceinline__ f32x4 *stage_at(uint8_t *stage, int c, int p) {
    return (f32x4 *)(stage + c * D * 4 + 16 * (p ^ (c & 15)));
}
template <int FMT, int D>
__device__ __forceinline__ void stage_o(uint8_t *stage, const State<FMT, D> &st) {
    const int ln = __lane_id(), j = ln & 31, h = ln >> 5;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const f32x4 x = {st.o[t][4 * a], st.o[t][4 * a + 1], st.o[t][4 * a + 2], st.o[t][4 * a + 3]};
            *stage_at<D>(stage, j, 8 * t + 2 * a + h) = x;
        }
}
// Where a column's outputs go, and what its sums are to be multiplied by: row (-1: nowhere), head.
struct Dest {
    int row, head;
    float f;
    int pad;
};
// The statistics of column R (m, l: of all its entries here), written; its sums' destination.
__device__ __forceinline__ Dest finish_column(const AttendArgs &A, int R, int cols, int row0, int hk, int split, float m,
                                              float l) {
    Dest d{-1, 0, 1.f, 0};
    if (R >= cols) return d;
    const int i = R / A.G;
    d.row = row0 + i;
    d.head = hk * A.G + (R - i * A.G);
    const int64_t rh = (int64_t)d.row * A.n_heads + d.head;
    if (A.splits > 1) {
        A.part_ml[(int64_t)split * A.T * A.n_heads + rh] = make_float2(m, l);
    } else {
        d.f = l == 0.f ? 0.f : 1.f / l;
        if (A.lse) A.lse[rh] = l == 0.f ? kNegInf : m * A.scale + kLn2 * __builtin_amdgcn_logf(l);
    }
    return d;
}
// Four values of N columns each: all the LDS they come from is read before the first store.
template <int FMT, int D, int N>
__device__ __forceinline__ void emit(const AttendArgs &A, const Dest (&d)[N], int split, int piece, const f32x4 (&o)[N]) {
    if (A.splits > 1) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            if (d[n].row >= 0)
                *(f32x4 *)(A.part_o + (((int64_t)split * A.T + d[n].row) * A.n_heads + d[n].head) * D + 4 * piece) = o[n];
        return;
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int64_t at = d[n].row * A.out_ld + d[n].head * D + 4 * piece;
        const f32x4 x = o[n] * d[n].f;
        if (d[n].row < 0) continue;
        if constexpr (FMT == KEY_F32) *(f32x4 *)((float *)A.out + at) = x;
        else *(u32x2 *)((uint16_t *)A.out + at) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
    }
}
// A wave's 32 columns from c on, staged in LDS by itself: all of them out.
template <int FMT, int D>
__device__ __forceinline__ void emit_columns(const AttendArgs &A, const State<FMT, D> &st, int c, int cols, int row0,
                                             int hk, int split, uint8_t *stage, Dest *dest) {
    constexpr int P = D / 4, PER = 64 / P, N = 4;         // pieces of a column, columns at once
    const int ln = __lane_id();
    const float l = both_sum(st.l);
    if (ln < 32) dest[ln] = finish_column(A, c + ln, cols, row0, hk, split, st.m, l);
    stage_o<FMT, D>(stage, st);
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int e = ln / P; e < 32; e += N * PER) {
        Dest d[N];
        f32x4 o[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            d[n] = dest[e + n * PER];
            o[n] = *stage_at<D>(stage, e + n * PER, ln % P);
        }
        emit<FMT, D, N>(A, d, split, ln % P, o);
    }
}

// ------------------------------------------------------------------ few columns
// Workgroup (split, kv head, request), at most 32 columns: its tiles are dealt to the four waves
// in turn.  bf16 and float32 tiles are copied straight into the wave's own LDS: the next keys' copy
// is issued once the scores are formed and the next values' once they are weighed, so each wave
// has one to two copies in flight and waits for no other wave.  fp8 tiles are loaded a tile ahead
// into registers.  Bound by memory: one token of 32 requests x 32 heads over 4,096 entries 100 us,
// 5.5 TB/s (a large copy: 4.84 TB/s read and written); of 30 over 32,768 fp8 entries 387 us, 5.3
// TB/s; one token of one request 8 us, a launch and the chain of its first loads.
template <int FMT, int D>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1)))
void attend_split_kernel(AttendArgs A) {
    using TL = Tile<FMT, D>;
    constexpr bool FP8 = FMT == KEY_FP8;
    constexpr int NI = TL::BYTES / 1024;
    __shared__ __align__(16) uint8_t sK[4][TL::BYTES], sV[FP8 ? 1 : 4][FP8 ? 16 : TL::BYTES];
    __shared__ float sS[FP8 ? 4 : 1][2][64], sM[4][32], sL[4][32];
    __shared__ Dest sE[32];
    __shared__ Special<D> sX[4];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), ln = __lane_id(), j = ln & 31;
    const int split = blockIdx.x % A.splits, hk = (blockIdx.x / A.splits) % A.n_kv, b = blockIdx.x / (A.splits * A.n_kv);
    const Req rq = request(A, b);
    const int cols = rq.n * A.G;
    if (cols == 0) return;
    const Span sp = make_span<TL::E>(A, 0, rq.n - 1, rq.n, rq.len);
    const int per = (sp.count + A.splits - 1) / A.splits;
    const int t0 = split * per + w, t1 = min(sp.count, (split + 1) * per);
    const uint8_t *kp = (const uint8_t *)A.k, *vp = (const uint8_t *)A.v;
    const uint32_t key0 = key_lane<FMT, D>(), value0 = value_lane<FMT, D>();
    uint8_t *kt = sK[w], *vt = FP8 ? sK[w] : sV[FP8 ? 0 : w];
    // the next mapped tile from i on, and its page (i >= t1: none)
    int page = -1;
    auto seek = [&](int i) {
        page = -1;
        for (; i < t1; i += 4) {
            page = __builtin_amdgcn_readfirstlane(page_of<FMT, D>(A, b, sp.at(i)));
            if (page >= 0) break;
        }
        return i;
    };
    CodeRegs<FP8 ? 8 : 1> kc, vc;
    auto issue_k = [&](int t) {
        const uint8_t *src = kp + tile_at<FMT, D>(A, page, hk, t);
        if constexpr (FP8) load_codes<8, 64>(kc, src, again(ln));
        else {
#pragma unroll
            for (int n = 0; n < NI; ++n) copy_pieces<FMT, D, true>(src, kt, n);
        }
    };
    auto issue_v = [&](int t) {
        const uint8_t *src = vp + tile_at<FMT, D>(A, page, hk, t);
        if constexpr (FP8) load_codes<8, 64>(vc, src, again(ln));
        else {
#pragma unroll
            for (int n = 0; n < NI; ++n) copy_pieces<FMT, D, false>(src, vt, n);
        }
    };
    int i = seek(t0);
    if (i < t1) {
        issue_k(sp.at(i));
        issue_v(sp.at(i));
    }
    const Col col = make_col(A, j, rq.row0, rq.n, rq.len);
    u32x4 q[TL::QR];
    State<FMT, D> st;
    load_q<FMT, D>(q, A, j, rq.row0, hk, col.valid);
    st.clear();
    clear_special(sX[w]);
    while (i < t1) {
        const int t = sp.at(i), s0 = t * TL::E;
        const int nx = seek(i + 4);
        const uint32_t me = again(ln), klane = again(key0), vlane = again(value0);
        if constexpr (FP8) {
            put_codes<8, 64, true>(kc, kt, sS[w][0], me, as_is);
            __builtin_amdgcn_wave_barrier();
        } else {
            wait_vm<NI>();                                // the keys; the values may be in flight
        }
        f32x16 s[TL::SUB];
#pragma unroll
        for (int sub = 0; sub < TL::SUB; ++sub) s[sub] = scores<FMT, D>(kt, klane, sub, q);
        __builtin_amdgcn_s_waitcnt(0xc07f);               // lgkmcnt(0): the keys are read
        __builtin_amdgcn_sched_barrier(0);
        if (nx < t1) issue_k(sp.at(nx));
        if constexpr (FP8) {
            put_codes<8, 64, false>(vc, vt, sS[w][1], me, as_is);
            __builtin_amdgcn_wave_barrier();
            if (nx < t1) issue_v(sp.at(nx));
        }
        constexpr uint64_t full = ~0ull >> (64 - TL::E);
        const uint64_t vis = col.valid ? visible(col, s0, A.mask_ld) & full : full;
        const bool masked = __ballot(vis != full) != 0;
        soften<FMT, D, TL::SUB>(s, masked, vis, A.c, sS[FP8 ? w : 0][0], sS[FP8 ? w : 0][1], st);
        if constexpr (!FP8) {
            if (nx < t1) wait_vm<NI>();                   // the values; the next keys may be in flight
            else wait_vm<0>();
        }
        add_values<FMT, D, TL::SUB>(vt, vlane, s, masked && any_special<FMT, D>(vt), vis, st, sX[w]);
        __builtin_amdgcn_s_waitcnt(0xc07f);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!FP8) {
            if (nx < t1) issue_v(sp.at(nx));
        }
        i = nx;
    }
    // the four waves' parts, joined and written by all threads
    const float l = both_sum(st.l);
    if (ln < 32) {
        sM[w][j] = st.m;
        sL[w][j] = l;
    }
    apply_special<FMT, D>(sX[w], st);
    stage_o<FMT, D>(kt, st);
    __syncthreads();
    if (tid < 32) {
        float m = kNegInf, sum = 0.f, f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) m = fmaxf(m, sM[k][tid]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = sM[k][tid] == kNegInf ? 0.f : __builtin_amdgcn_exp2f((sM[k][tid] - m) * A.c);
            sum += f[k] * sL[k][tid];
        }
        sE[tid] = finish_column(A, tid, cols, rq.row0, hk, split, m, sum);
#pragma unroll
        for (int k = 0; k < 4; ++k) sM[k][tid] = f[k];
    }
    __syncthreads();
    constexpr int P = D / 4, N = 32 * P / 256;
    Dest d[N];
    f32x4 o[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = tid / P + n * (256 / P);
        d[n] = sE[c];
        o[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n] += sM[k][c] * *stage_at<D>(sK[k], c, tid % P);
    }
    emit<FMT, D, N>(A, d, split, tid % P, o);
}

// A workgroup's part of the entries, block of columns, kv head and request.  Consecutive workgroups
// run on the chip's 8 XCDs in turn, each with an L2 of its own: with the kv heads innermost, those
// of one head share an XCD.  Blocks differ in their tiles, which the host does not know; where that
// matters (ranked) each workgroup ranks them for itself, and the longest go first, so that the
// short ones even out the end.
struct Place {
    int split, blk, hk, b;
};
template <int E, int COLS>
__device__ __forceinline__ Place place_of(const AttendArgs &A, int *ranked) {   // kAttendRanked + 4
    const int hk = blockIdx.x % A.n_kv, n = blockIdx.x / A.n_kv, split = n % A.splits, rank = n / A.splits;
    const int items = A.B * A.blocks, tid = threadIdx.x;
    int it = items - 1 - rank;                            // later blocks see more entries
    if (A.ranked) {
        int own = -1;
        if (tid < items) {
            const int b = tid / A.blocks, c0 = (tid - b * A.blocks) * COLS;
            const Req rq = request(A, b);
            const int cols = rq.n * A.G;
            own = 0;
            if (c0 < cols) own = 1 + make_span<E>(A, c0 / A.G, (min(c0 + COLS, cols) - 1) / A.G, rq.n, rq.len).count;
        }
        if (tid < kAttendRanked) ranked[tid] = own;
        __syncthreads();
        if (tid < items) {
            int before = 0;
            for (int k = 0; k < items; k += 4) {
                const int4 x = *(const int4 *)(ranked + k);
                before += (x.x > own || (x.x == own && k < tid)) + (x.y > own || (x.y == own && k + 1 < tid)) +
                          (x.z > own || (x.z == own && k + 2 < tid)) + (x.w > own || (x.w == own && k + 3 < tid));
            }
            if (before == rank) ranked[kAttendRanked] = tid;
        }
        __syncthreads();
        it = __builtin_amdgcn_readfirstlane(ranked[kAttendRanked]);
    }
    const int b = it / A.blocks;
    return {split, it - b * A.blocks, hk, b};
}

// ------------------------------------------------------------------ many columns, float32
// Workgroup (split, block of 128 columns, kv head, request) of four waves, 32 columns each; the
// 32-entry tiles are shared.  The next tile's copy (two LDS stages) is in flight while a tile is
// worked on, one barrier a tile.  Bound by the float32 MFMAs (154 TFLOP/s in a large product) and,
// with one workgroup a CU, by the latency from scores to sums: 5.3 to 5.8 us a tile of 32 entries
// of 128 dims either way.  3 requests of up to 333 rows x 12 heads of 64 dims: 25 us and 5 us to join.
template <int D>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void attend_tile_kernel(AttendArgs A) {
    constexpr int FMT = KEY_F32;
    using TL = Tile<FMT, D>;
    constexpr int NI = TL::BYTES / 4096;                  // copy instructions a wave and tile
    __shared__ __align__(16) uint8_t sK0[TL::BYTES], sV0[TL::BYTES], sK1[TL::BYTES], sV1[TL::BYTES];
    __shared__ Special<D> sX[4];
    __shared__ Dest sE[4][32];
    __shared__ __align__(16) int sP[kAttendRanked + 4];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), ln = __lane_id(), j = ln & 31;
    const Place at = place_of<TL::E, 128>(A, sP);
    const int split = at.split, blk = at.blk, hk = at.hk, b = at.b;
    const Req rq = request(A, b);
    const int cols = rq.n * A.G, c0 = blk * 128;
    if (c0 >= cols) return;
    const Span sp = make_span<TL::E>(A, c0 / A.G, (min(c0 + 128, cols) - 1) / A.G, rq.n, rq.len);
    const int per = (sp.count + A.splits - 1) / A.splits;
    const int t0 = split * per, t1 = min(sp.count, t0 + per);
    const int R = c0 + 32 * w + j;
    const bool idle = c0 + 32 * w >= cols;
    Col col;
    u32x4 q[TL::QR];
    State<FMT, D> st;
    const uint32_t key0 = key_lane<FMT, D>(), value0 = value_lane<FMT, D>();
    const uint8_t *kp = (const uint8_t *)A.k, *vp = (const uint8_t *)A.v;
    int page = -1;
    auto seek = [&](int i) {
        page = -1;
        for (; i < t1; ++i) {
            page = __builtin_amdgcn_readfirstlane(page_of<FMT, D>(A, b, sp.at(i)));
            if (page >= 0) break;
        }
        return i;
    };
    auto issue = [&](uint8_t *kt, uint8_t *vt, int t) {
        const int64_t ofs = tile_at<FMT, D>(A, page, hk, t);
#pragma unroll
        for (int n = 0; n < NI; ++n) copy_pieces<FMT, D, true>(kp + ofs, kt, NI * w + n);
#pragma unroll
        for (int n = 0; n < NI; ++n) copy_pieces<FMT, D, false>(vp + ofs, vt, NI * w + n);
    };
    auto work = [&](const uint8_t *kt, const uint8_t *vt, int t) {
        constexpr uint64_t full = ~0ull >> (64 - TL::E);
        const uint64_t vis = col.valid ? visible(col, t * TL::E, A.mask_ld) & full : full;
        if (idle || __builtin_amdgcn_ballot_w64(col.valid && vis != 0) == 0) return;
        const bool masked = __builtin_amdgcn_ballot_w64(vis != full) != 0;
        SRegs<1> s;
        s[0] = scores<FMT, D>(kt, again(key0), 0, q);
        soften<FMT, D, 1>(s, masked, vis, A.c, nullptr, nullptr, st);
        add_values<FMT, D, 1>(vt, again(value0), s, masked && any_special<FMT, D>(vt), vis, st, sX[w]);
    };
    int i = seek(t0);
    // tile i is on its way to (kt, vt); after the barrier the other stage is free for the next
    auto step = [&](uint8_t *kt, uint8_t *vt, uint8_t *kn, uint8_t *vn) {
        const int t = sp.at(i);
        wait_vm<0>();
        __syncthreads();
        i = seek(i + 1);
        if (i < t1) issue(kn, vn, sp.at(i));
        work(kt, vt, t);
    };
    if (i < t1) issue(sK0, sV0, sp.at(i));
    col = make_col(A, R, rq.row0, rq.n, rq.len);          // beside the first tile's copy
    load_q<FMT, D>(q, A, R, rq.row0, hk, col.valid);
    st.clear();
    clear_special(sX[w]);
    while (i < t1) {
        step(sK0, sV0, sK1, sV1);
        if (i >= t1) break;
        step(sK1, sV1, sK0, sV0);
    }
    __syncthreads();
    apply_special<FMT, D>(sX[w], st);
    emit_columns<FMT, D>(A, st, c0 + 32 * w, cols, rq.row0, hk, split, w == 0 ? sK0 : w == 1 ? sV0 : w == 2 ? sK1 : sV1, sE[w]);
}

// ------------------------------------------------------------------ many columns, bf16 and fp8
// Workgroup (split, block of 256 columns, kv head, request) of eight waves, bf16 and fp8 caches.
// Each wave keeps the matrix unit busy with its own instructions: while a 32-entry tile's
// exponentials are formed, the next tile's scores run, and while its values are weighed, the next
// scores' mask and maximum.  Tiles pass through registers (loaded a tile ahead) into three LDS
// stages, with one barrier a 64-entry tile: when all waves have met in tile i, tile i + 1 is
// there and the stage of tile i - 1 is free.  (Copied straight into LDS they cost 3 to 5% more:
// prefill 287 / 296 us, ragged batch 460 / 481 us; the swizzle is then the source address's, a lane.)
//
// Bound by instruction issue and by the clock under this load (1.9 GHz; the same prefill over zeros
// takes 258 us instead of 296): the MFMAs are busy 44% of the cycles and the vector units 47%, half
// of the former beside the latter; the rest is the maximum's lane swap and branch, the barrier
// (without it, in a timing copy, 262 of 315 us) and waits for LDS.  4,096 rows x 32 heads
// under a window: 290 us, 949 TFLOP/s (a large bf16 product: 1,236).  8 ragged requests over 8,192
// entries 455 us, 910 TFLOP/s.  fp8 also widens codes and multiplies two scales: 30 trees of 64
// drafts over up to 24,576 entries 870 us, 770 TFLOP/s, on 240 of 256 CUs.
constexpr int kBlockNT = 512;
template <int FMT, int D>
struct Staged {
    using TL = Tile<FMT, D>;
    static constexpr int N = TL::BYTES / (16 * kBlockNT);   // 16-byte pieces a thread
    u32x4 k[N], v[N];
    __device__ __forceinline__ void load(const uint8_t *kp, const uint8_t *vp, int tid) {
#pragma unroll
        for (int n = 0; n < N; ++n) k[n] = *(const u32x4 *)(kp + 16 * kBlockNT * n + 16u * (uint32_t)tid);
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = *(const u32x4 *)(vp + 16 * kBlockNT * n + 16u * (uint32_t)tid);
    }
    // fix(row, piece, values): what is written of a piece of values
    template <class F>
    __device__ __forceinline__ void put(uint8_t *kt, uint8_t *vt, float *, float *, int tid, F fix) const {
        // a round of pieces is 32 or 64 rows: the swizzle repeats
        const uint32_t t = again(tid);
        const int r = t / TL::NP, at = t % TL::NP;
        const uint32_t ko = r * TL::ROW + 16 * (at ^ TL::swz_k(r)), vo = r * TL::ROW + 16 * (at ^ TL::swz_v(r));
#pragma unroll
        for (int n = 0; n < N; ++n) *(u32x4 *)(kt + ko + 16 * kBlockNT * n) = k[n];
#pragma unroll
        for (int n = 0; n < N; ++n) *(u32x4 *)(vt + vo + 16 * kBlockNT * n) =
            fix(r + kBlockNT / TL::NP * n, at, v[n], 1.f);
    }
};
template <>
struct Staged<KEY_FP8, kDim> {
    CodeRegs<1> k, v;
    __device__ __forceinline__ void load(const uint8_t *kp, const uint8_t *vp, int tid) {
        const uint32_t t = again(tid);
        load_codes<1, kBlockNT>(k, kp, t);
        load_codes<1, kBlockNT, true>(v, vp, t);
    }
    template <class F>
    __device__ __forceinline__ void put(uint8_t *kt, uint8_t *vt, float *ks, float *vs, int tid, F fix) const {
        const uint32_t t = again(tid);
        put_codes<1, kBlockNT, true>(k, kt, ks, t, as_is);
        put_codes<1, kBlockNT, false, true>(v, vt, vs, t, fix);
    }
};

template <int FMT, int D>
__global__ __launch_bounds__(kBlockNT) __attribute__((amdgpu_waves_per_eu(2, 2)))
void attend_block_kernel(AttendArgs A) {
    using TL = Tile<FMT, D>;
    constexpr bool FP8 = FMT == KEY_FP8;
    constexpr int S = 3, NW = kBlockNT / 64;
    static_assert(TL::SUB == 2, "two 32-entry tiles a tile");
    __shared__ __align__(16) uint8_t sK[S][TL::BYTES], sV[S][TL::BYTES];
    __shared__ float sS[FP8 ? S : 1][2][64];
    __shared__ Special<D> sX[NW];
    __shared__ Dest sE[NW][32];
    __shared__ __align__(16) int sP[kAttendRanked + 4];
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), ln = __lane_id(), j = ln & 31;
    const Place at = place_of<TL::E, 256>(A, sP);
    const int split = at.split, blk = at.blk, hk = at.hk, b = at.b;
    const Req rq = request(A, b);
    const int cols = rq.n * A.G, c0 = blk * 256;
    if (c0 >= cols) return;
    const Span sp = make_span<TL::E>(A, c0 / A.G, (min(c0 + 256, cols) - 1) / A.G, rq.n, rq.len);
    const int per = (sp.count + A.splits - 1) / A.splits;
    const int t0 = split * per, t1 = min(sp.count, t0 + per);
    const bool idle = c0 + 32 * w >= cols;
    const int R0 = c0 + 32 * w + j;
    const Col col = make_col(A, R0, rq.row0, rq.n, rq.len);
    u32x4 q[TL::QR];
    load_q<FMT, D>(q, A, R0, rq.row0, hk, col.valid);
    State<FMT, D> st;
    st.clear();
    clear_special(sX[w]);
    __syncthreads();                                       // marks may come from any wave

    // the next mapped tile from i on: its entries' places in the pools, and its index (i >= t1: none)
    constexpr int row = FP8 ? kRowFp8 : TL::ROW;
    const int64_t head = (int64_t)hk * kPage * row, step = (int64_t)A.n_kv * kPage * row;
    const uint8_t *kp = (const uint8_t *)A.k + head, *vp = (const uint8_t *)A.v + head;
    Staged<FMT, D> in;
    // a lane has the page of a tile: 64 at once, so that no tile waits for the table
    int first = t0, pages = t0 + ln < t1 ? page_of<FMT, D>(A, b, sp.at(t0 + ln)) : -1;
    auto fetch = [&](int i) {
        for (; i < t1; ++i) {
            if (i - first >= 64) {
                first = i;
                pages = i + ln < t1 ? page_of<FMT, D>(A, b, sp.at(i + ln)) : -1;
            }
            const int page = __builtin_amdgcn_readlane(pages, i - first);
            if (page < 0) continue;
            const int64_t at = page * step;
            in.load(kp + at, vp + at, tid);
            break;
        }
        return i;
    };

    // Tiles that some column of the workgroup sees only in part: masks are formed for these alone,
    // and their values that are not finite are kept out of LDS (a product with a masked entry's 0
    // would make them NaN): the thread that stages such a value marks the columns that see it.
    const int i0 = c0 / A.G, i1 = (min(c0 + 256, cols) - 1) / A.G, base = rq.len - rq.n;
    const int last = A.tree_mask ? rq.len : base + i1, from = max(last, 0) - (A.window - 1);   // all see [from, upto)
    const int upto = max(0, A.tree_mask ? base : base + i0 + 1), most = A.tree_mask ? rq.len : base + i1 + 1;
    const int whole0 = min(A.n_sink, upto) / TL::E;        // tiles [0, whole0) and [whole1, whole2) are seen whole
    const int whole1 = tiles_of<TL::E>(max(from, 0)), whole2 = upto / TL::E;
    auto put = [&](int s, int t, bool edge) {
        uint8_t *kt = sK[s], *vt = sV[s];
        float *ks = sS[FP8 ? s : 0][0], *vs = sS[FP8 ? s : 0][1];
        if (!edge) {
            in.put(kt, vt, ks, vs, tid, as_is);
            return;
        }
        in.put(kt, vt, ks, vs, tid, [&](int r, int piece, u32x4 y, float scale) {
            const bool wild = !(fabsf(scale) < __builtin_inff());
            uint32_t bad = wild;
#pragma unroll
            for (int d = 0; d < 4; ++d) bad |= ((y[d] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
            if (bad == 0) return y;
            const int entry = t * TL::E + r;
#pragma unroll 1
            for (int c = 0; c < 256 && entry < most; ++c) {
                const Col k = make_col(A, c0 + c, rq.row0, rq.n, rq.len);
                if (!k.valid || !(visible(k, t * TL::E, A.mask_ld) >> r & 1)) continue;
                Special<D> &x = sX[c / 32];
                x.any = 1;
#pragma unroll 1
                for (int e = 0; e < 8; ++e) {
                    const uint32_t word = e < 2 ? y[0] : e < 4 ? y[1] : e < 6 ? y[2] : y[3];
                    uint32_t f = e & 1 ? word & 0xffff0000u : word << 16;
                    if constexpr (FP8) f = __float_as_uint(__uint_as_float(f) * scale);
                    if ((f & 0x7f800000u) != 0x7f800000u) continue;
                    uint32_t *to = f & 0x007fffffu ? x.nan[c % 32] : f >> 31 ? x.down[c % 32] : x.up[c % 32];
                    atomicOr(&to[piece / 4], 1u << (8 * (piece % 4) + e));
                }
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) y[d] = wild ? 0u : finite_only<false>(y[d]);
            return y;
        });
        if constexpr (FP8) {                               // those values are zeros: any scale will do
            if ((tid & 7) == 0 && !(fabsf(in.v.scale) < __builtin_inff())) vs[tid >> 3] = 0.f;
        }
    };

    // the scores of the 32-entry tile being worked on and of the next; the mask of their tile
    SRegs<1> sa, sb;
    uint64_t vis = ~0ull;
    bool masked = false;
    auto set_mask = [&](int t, bool edge) {
        masked = false;
        if (!edge) return;
        vis = col.valid ? visible(col, t * TL::E, A.mask_ld) : ~0ull;
        masked = __builtin_amdgcn_ballot_w64(vis != ~0ull) != 0;
    };
    // Scores formed (and, fp8, scaled) with their maximum mx; a mask changes both.
    auto settle = [&](SRegs<1> &s, int sub, float mx) {
        if (masked) {
            hide<1>(s, vis >> (32 * sub));
            mx = max_of<1>(s);
        }
        raise_max<FMT, D>(mx, A.c, st);
    };
    // The exponentials of one 32-entry tile beside the scores of the next, then its values; returns
    // the scores' maximum.  Written in the order it is to run in, a matrix instruction and what
    // fits beside it at a time.  The keys are read before the step that uses them (read_keys), behind
    // the maximum's lane swap and branch.
    uint32_t ko[TL::QR], vo[TL::DT];                      // the lane's reads in the current stages
#pragma unroll
    for (int i = 0; i < TL::QR; ++i) ko[i] = key_lane<FMT, D>() ^ (uint32_t)(32 * i);
#pragma unroll
    for (int t = 0; t < TL::DT; ++t) vo[t] = value_lane<FMT, D>() ^ (uint32_t)(64 * t);
    auto move_keys = [&](int by) {
#pragma unroll
        for (int i = 0; i < TL::QR; ++i) ko[i] += (uint32_t)by;
    };
    auto move_values = [&](int by) {
#pragma unroll
        for (int t = 0; t < TL::DT; ++t) vo[t] += (uint32_t)by;
    };
    u32x4 ka[TL::QR];
    auto read_keys = [&](int sub) {
#pragma unroll
        for (int i = 0; i < TL::QR; ++i) ka[i] = *(const u32x4 *)(sK[0] + 32 * sub * TL::ROW + ko[i]);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto advance = [&](SRegs<1> &now, int stage, int sub, SRegs<1> &then, int stage2, int sub2) {
        const uint8_t *vt = sV[0] + 32 * sub * TL::ROW;
        constexpr int QR = TL::QR;                        // matrix instructions of each product
        static_assert(QR == 2 * TL::DT, "as many of each");
        u32x4 va[2][TL::DT];
        u32x2 pk[2][2];
        // fp8 scales of four entries at a time, read a step or two before they are used
        f32x4 four[2];
        auto read_scales = [&](int a, const float *from) {
            if constexpr (FP8) four[a & 1] = *(const f32x4 *)(from + 8 * a + 4 * (ln >> 5));
        };
        read_scales(0, sS[FP8 ? stage : 0][1] + 32 * sub);
        float sum = st.l;
        // the products go before the other wave's staging and maxima (without: prefill 303 / 296 us,
        // ragged batch 466 / 455 us, 64-draft fp8 trees 894 / 883 us)
        __builtin_amdgcn_s_setprio(1);
        f32x16 s;
#pragma unroll
        for (int v = 0; v < 16; ++v) s[v] = 0.f;
        auto read_values = [&](int x) {                   // k step x / DT, values 32 (x % DT) and on
            const uint8_t *row = vt + vo[x % TL::DT] + 16 * (x / TL::DT) * TL::ROW;
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)row));
            const u32x2 c = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4 *)(row + 8 * TL::ROW)));
            va[x / TL::DT][x % TL::DT] = u32x4{a[0], a[1], c[0], c[1]};
        };
        auto raise = [&](int v) {                         // entries v, v + 1
            if (v % 4 == 0 && v < 12) read_scales(v / 4 + 1, sS[FP8 ? stage : 0][1] + 32 * sub);
            if (v == 14) read_scales(0, sS[FP8 ? stage2 : 0][0] + 32 * sub2);
            float p0 = __builtin_amdgcn_exp2f(fmaf(now[0][v], A.c, -st.mc));
            float p1 = __builtin_amdgcn_exp2f(fmaf(now[0][v + 1], A.c, -st.mc));
            sum += p0;
            sum += p1;
            if constexpr (FP8) {
                p0 *= four[v / 4 & 1][v % 4];
                p1 *= four[v / 4 & 1][v % 4 + 1];
            }
            pk[v / 8][v % 8 / 4][v % 4 / 2] = pack_bf16(p0, p1);
        };
        auto weigh_one = [&](int x) {
            const u32x4 b = {pk[x / TL::DT][0][0], pk[x / TL::DT][0][1], pk[x / TL::DT][1][0], pk[x / TL::DT][1][1]};
            st.o[x % TL::DT] = mma_bf16(va[x / TL::DT][x % TL::DT], b, st.o[x % TL::DT]);
        };
        // half of the scores, with the first k step's exponentials
        constexpr int DT = TL::DT;
#pragma unroll
        for (int i = 0; i < DT; ++i) {
            s = mma_bf16(ka[i], q[i], s);
            read_values(i);
#pragma unroll
            for (int v = 8 / DT * i; v < 8 / DT * (i + 1); v += 2) raise(v);
            here(sum);
            __builtin_amdgcn_sched_barrier(0);
        }
        // the other half in turn with that step's values, and the second step's exponentials
#pragma unroll
        for (int i = 0; i < DT; ++i) {
            weigh_one(i);
            read_values(DT + i);
            raise(8 + 8 / DT * i);
            here(sum);
            __builtin_amdgcn_sched_barrier(0);
            s = mma_bf16(ka[DT + i], q[DT + i], s);
            if constexpr (DT == 2) raise(10 + 4 * i);
            here(sum);
            __builtin_amdgcn_sched_barrier(0);
        }
        st.l = sum;
        // the second step's values, with the scores' scales and maximum
        float mx = kNegInf;
        constexpr int MX = 16 / DT;
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            weigh_one(DT + x);
#pragma unroll
            for (int v = MX * x; v < MX * (x + 1); ++v) {
                if (v % 4 == 0 && v < 12) read_scales(v / 4 + 1, sS[FP8 ? stage2 : 0][0] + 32 * sub2);
                if constexpr (FP8) s[v] *= four[v / 4 & 1][v % 4];
                mx = fmaxf(mx, s[v]);
            }
            here(mx);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
        then[0] = s;
        return mx;
    };
    // A wave without columns runs the same loop, copying its share of the tiles.
    auto run = [&](auto active) {
        constexpr bool on = decltype(active)::value;
        auto is_edge = [&](int t) { return t >= whole0 && (t < whole1 || t >= whole2); };
        int i = fetch(t0), stage = 0;
        if (i >= t1) return;
        int t = sp.at(i);
        bool edge = is_edge(t);
        put(0, t, edge);
        i = fetch(i + 1);                                  // the tile on its way
        __syncthreads();
        if constexpr (on) {
            sa[0] = scores<FMT, D>(sK[0], key_lane<FMT, D>(), 0, q);
            if constexpr (FP8) scale_scores<1>(sa, sS[0][0]);
            set_mask(t, edge);
            settle(sa, 0, max_of<1>(sa));
            read_keys(1);
        }
        bool more;
        do {
            const int next = stage == S - 1 ? 0 : stage + 1, by = (next - stage) * TL::BYTES;
            more = i < t1;
            float mx = 0.f;
            if constexpr (on) mx = advance(sa, stage, 0, sb, stage, 1);
            if (more) {
                t = sp.at(i);
                edge = is_edge(t);
                put(next, t, edge);
                i = fetch(i + 1);
                __syncthreads();
            }
            if constexpr (on) {
                move_keys(by);
                read_keys(0);
                settle(sb, 1, mx);
                mx = advance(sb, stage, 1, sa, next, 0);
                move_values(by);
                read_keys(1);
                set_mask(t, edge && more);
                if (!more) mx = kNegInf;                   // scores of no tile: they raise nothing
                settle(sa, 0, mx);
            }
            stage = next;
        } while (more);
    };
    if (idle) run(std::false_type());
    else run(std::true_type());
    // outputs through LDS, a stage for a wave's 32 columns, four waves at a time
    static_assert(32 * D * 4 == TL::BYTES, "a stage holds a wave's outputs");
#pragma unroll 1
    for (int round = 0; round < NW / 4; ++round) {
        __syncthreads();
        if (idle || w / 4 != round) continue;
        apply_special<FMT, D>(sX[w], st);
        emit_columns<FMT, D>(A, st, c0 + 32 * w, cols, rq.row0, hk, split, w % 4 < 3 ? sK[w % 4] : sV[0], sE[w]);
    }
}

// ------------------------------------------------------------------ joining the parts
// One wave a (row, head): lane s weighs part s by e^(m - max), then each lane sums its D / 64
// values over the parts, eight parts' loads at a time.  16 parts of 64 columns: 4 us.
template <int FMT, int D>
__global__ __launch_bounds__(256) void attend_merge_kernel(AttendArgs A) {
    constexpr int W = D / 64;
    const int ln = __lane_id();
    const Req rq = request(A, blockIdx.y);
    const int64_t e = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int i = (int)(e / A.n_heads), head = (int)(e % A.n_heads);
    if (i >= rq.n) return;
    const int64_t row = rq.row0 + i, rh = row * A.n_heads + head, all = (int64_t)A.T * A.n_heads;
    const float2 x = ln < A.splits ? A.part_ml[ln * all + rh] : make_float2(kNegInf, 0.f);
    float m = x.y == 0.f ? kNegInf : x.x;                 // a part that saw nothing left no sums
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float f = x.y == 0.f || x.x == kNegInf ? 0.f : __builtin_amdgcn_exp2f((x.x - m) * A.c);
    float l = f * x.y;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) l += __shfl_xor(l, o);
    float o[W];
#pragma unroll
    for (int k = 0; k < W; ++k) o[k] = 0.f;
    const float *src = A.part_o + rh * D + W * ln;
    constexpr int U = 8;
    for (int s0 = 0; s0 < A.splits; s0 += U) {
        float v[U][W];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float *p = src + min(s0 + u, A.splits - 1) * all * D;
#pragma unroll
            for (int k = 0; k < W; ++k) v[u][k] = p[k];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float g = s0 + u < A.splits ? __shfl(f, s0 + u) : 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) o[k] += g == 0.f ? 0.f : g * v[u][k];
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = row * A.out_ld + (int64_t)head * D + W * ln;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        if constexpr (FMT == KEY_F32) ((float *)A.out)[at + k] = o[k] * inv;
        else ((uint16_t *)A.out)[at + k] = (uint16_t)pack_bf16(o[k] * inv, 0.f);
    }
    if (ln == 0 && A.lse) A.lse[rh] = l == 0.f ? kNegInf : m * A.scale + kLn2 * __builtin_amdgcn_logf(l);
}

template <int FMT, int D>
hipError_t launch(const AttendArgs &a, hipStream_t s) {
    const unsigned wgs = (unsigned)((int64_t)a.splits * a.n_kv * a.B * std::max(a.blocks, 1));
    if (a.blocks) {
        if constexpr (FMT == KEY_F32) attend_tile_kernel<D><<<dim3(wgs), 256, 0, s>>>(a);
        else attend_block_kernel<FMT, D><<<dim3(wgs), kBlockNT, 0, s>>>(a);
    } else {
        attend_split_kernel<FMT, D><<<dim3(wgs), 256, 0, s>>>(a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t waves = (int64_t)a.max_rows * a.n_heads;
    attend_merge_kernel<FMT, D><<<dim3((unsigned)((waves + 3) / 4), (unsigned)a.B), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int attend_tile_entries(int key_fmt) { return key_fmt == KEY_F32 ? 32 : 64; }
int attend_block_columns(int key_fmt) { return key_fmt == KEY_F32 ? 128 : 256; }

hipError_t launch_attend(const AttendArgs &a, int key_fmt, int head_dim, hipStream_t s) {
    if (key_fmt == KEY_F32) return head_dim == 64 ? launch<KEY_F32, 64>(a, s) : launch<KEY_F32, 128>(a, s);
    if (key_fmt == KEY_BF16) return head_dim == 64 ? launch<KEY_BF16, 64>(a, s) : launch<KEY_BF16, 128>(a, s);
    return launch<KEY_FP8, kDim>(a, s);
}

}  // namespace fm
