// tree.cu -- attention of a tree of drafted tokens over the paged cache.
//
// Request r has q_len drafted tokens, already written to its pages as the
// last q_len of its L positions; ctx = L - q_len.  Draft i sees context key
// j < ctx, and draft key ctx + n iff bit n of its mask is set:
//   pos(j) = j for a context key, ctx + depth[n] for draft key n
//   keep key j iff visible and (window_left < 0 or pos(j) >= qpos - window_left),
//   qpos = ctx + depth[i]
//   s = sm_scale * <q, k_j> + alibi[h] * (pos(j) - qpos);  o = softmax(s, sink) V.
//
// What bounds it: a decode step with q_len queries reads K and V once, so up
// to about 128 rows (drafts x heads of a group) per kv head it is HBM bound;
// beyond that the tensor cores are.  mma.sync would be the limit from 64 rows
// on, so the products run on tcgen05: the (draft, head) rows of one kv head are
// packed into tiles of 128 rows (M = 128), and because a 128-key step costs
// the tensor core about half the time its 64 KB of bf16 K and V take from HBM,
// the padding of small trees is free.
//
// Over 8-bit pools the codes become f16 tiles, each row times 2^(its scale's
// exponent - the tile's largest), which is exact while the tile's scales lie within
// 2^15 of one another.  The tile's two largest scales are scalars of the softmax:
// K's multiplies the scores, V's moves the exponent of the weights.  Where a tile's
// scales are wider apart than kSpreadK or kSpreadV (a hidden draft may hold
// anything), its rows stay as the codes are, and the softmax takes the scale
// bytes key by key: exact too, and slower.  So a key that a draft does not see
// never costs it bits, and one that it hardly weighs next to none (kSpreadV).  q is scaled per row by a power of two into f16 (decode_fp8.cu gives
// the error bound).
//
// Persistent CTAs, one per SM, in groups of one CTA per kv head.  The work of a kv
// head is one line of key tiles: request after request, and in a request row
// group after row group (X row tiles of one request; its key tiles).  Group i
// takes the i-th equal part of the line, so every SM is busy to the end
// whatever the lengths are, and a CTA's fixed costs (Q, the pipeline's fill, the
// last rows out) come once per row group it meets, with the next K and V tiles
// already on their way.  A row group that lies in one group's part is stored by
// it; one that is cut leaves partials, at most two per CTA, for a merge kernel.
// The heads of one group read the same tokens at the same time.
//
// Warps: four softmax warps per row tile, one row per thread; a TMA warp, which
// also works out the CTA's segments and hands them to the others through a
// ring; an MMA warp; over 8-bit pools the warps that convert codes, K's beside V's
// (one after the other: 10 % more for 8 x 32 drafts over 24K).
//   S = Q K^T -> TMEM; the softmax reads S twice (maximum, weights), writes P (16
//   bits) over S; O += P V with P from TMEM.  O is rescaled only when a row's
//   maximum has grown a lot.
// The products run in units n = (key tile, row tile), row tiles fastest, with two S
// buffers in turn: S(n + 2) is issued right behind O(n), so a unit's softmax
// always has the other buffer's products beside it -- those of the other row
// tile, or of the next key tile when there is one.  Two row tiles share every
// K and V tile.
// Tiles that hold anything a row does not see (the drafts, the window's edge,
// the ends of the partition) take a general path with visibility bits; V rows
// behind the end are zeroed, and a V row with a non-finite value is zeroed too
// and reaches, as NaN, only the rows that see it.
//
// P rounds to the operands' type: f16 over 8-bit pools, bf16 (half a step 2^-8) over
// bf16 ones, as in prefill.cu and decode.cu; the sum of the weights is of those not
// rounded.  Of the error against 64 bits, which the output's own rounding makes 0.0016
// of the outputs' size, that leaves 0.0017 on short contexts and 0.0023 on 16K..32K.
//
// Measured (GB300, 32/8 heads of 128): 8 x 64 drafts over 16K..32K tokens of bf16
// 185 us in a replayed graph and 194 as calls, 67 and 64 % of a copy's rate; 16 x 24
// over 0.5K..8K of the 8-bit cache 72 us, 27 %; 4 x 8 over 60..900 of bf16 16 us, mostly
// the latency of two kernels.  With one row tile and 32-token pages, 8 x 32 over 24K
// takes 137 us, 87 %.
//   Two row tiles per CTA (X = 2, heads up to 128) when a request may have more
// than 128 rows: 8 x 64 drafts over 24K 175 us (8-bit: 239) against 255 (280) with
// one, which reads K and V twice; 8 x 40 drafts, whose second tile is a quarter
// full, 168 (225) against 249 (275).
//   Slower: K and V on their way to L2 two tiles before their loads (70 -> 77 us,
// 8-bit), fewer converted and more raw tiles (173 -> 198 us), eight converting
// warps (short cases 73 -> 76 us, long ones 153 -> 149).
//   What bounds it: with two row tiles 4 x 527 cycles of tensor work in about 4000
// per key tile, the rest handing S, P and O between the warps; over 8-bit pools
// the same hand-overs, the conversion's among them, about 3300 cycles per key
// tile (8 x 32 drafts over 24K: 151 us; by a probe some 20 less without the softmax's
// arithmetic, as many without the conversion's, 45 without either); and some 5 us per row group that
// a CTA meets, for Q, the general tile and code that is fetched for the first time.
#include "pkv_fp8.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kTile = 128;      // rows and keys per tile
constexpr int kRing = 4;        // segments handed over ahead
constexpr int kInfo = 8;        // key tiles whose bad pages are: more than are ever under way
constexpr int kPoison = 4;      // repaired tiles whose poison words are kept: as many as V tiles
constexpr float kNegInf = -INFINITY;
// A row's reference moves (and O is rescaled, which costs about a tile's time)
// only when a score exceeds it by kLazy log2 units.  bf16 weights have fp32's
// range and lose nothing by it; f16 weights start at 2^kWeightExp and stay
// below 2^15, with 11 bits kept down to 2^-20 of the reference and an error of
// 2^-31 of it below that.  With 4 for both, rows of real spread rescaled in half
// of the tiles: 402 us instead of 229 on 8 x 64 drafts over 16K..32K tokens.
template <bool KV8>
constexpr float kLazy = KV8 ? 9.f : 24.f;
constexpr int kWeightExp = 6;
// Over 8-bit pools the sum of the weights has a reference of its own, the row's
// largest score as of when it was last exceeded by this much (fp32 has the room).
constexpr float kLazySum = 60.f;
// How far apart (log2) a tile's scales may lie for its rows to share one.  K: a code's
// smallest step, 2^-9, times 2^-15 is f16's smallest number.  V: the same would be
// exact, but f16 weights count from the tile's largest scale, which the row's
// weightiest keys may not have: they lose kSpreadV of the 31 bits above.  8 x 32
// drafts over 24K take 151 us where no tile is wider (scales that vary by 2^N(0, 1)
// from row to row), 252 where 95 % of V's tiles are (2^N(0, 2)), and 500 where V's all
// are and half of K's (2^N(0, 3); K's take the general code).
constexpr int kSpreadK = 15, kSpreadV = 8;

// T: tile width (head size padded to 64, 128 or 256); X: row tiles per CTA.
template <int T, bool KV8, int X>
struct Cfg {
    static constexpr int HALVES = T / 64;
    static constexpr int HALF = kTile * 128;         // 128 rows of 64 dims
    static constexpr int TILE = HALVES * HALF;
    // K and V tiles: as many as fit, for the bytes in flight (over 8-bit pools the
    // raw tiles are what is in flight, and an f16 tile each way hides the
    // conversion; beside two row tiles one K and two V tiles take 241 us, two and
    // one 251, for 8 x 64 drafts over 24K)
    static constexpr int KB = KV8 ? (T == 64 || (T == 128 && X == 1) ? 2 : 1)
                                  : T == 64 ? 4 : T == 128 ? 3 : 1;
    static constexpr int VB = KV8 ? (T <= 128 ? 2 : 1)
                                  : T == 64 ? 4 : T == 128 ? 4 - X : 1;
    // raw tiles of codes, K and V in turn
    static constexpr int RU = !KV8 ? 0 : T == 256 ? 1 : 4;
    static constexpr int RAW = T * kTile;
    static constexpr int ROWB = T < 128 ? T : 128;   // bytes of a raw box row
    static constexpr int DW = !KV8 ? 0 : 4;        // converting warps
    // K and V are converted side by side, each by half of them, unless both pass
    // through one raw tile
    static constexpr bool SPLIT = KV8 && RU > 1;
    static constexpr int FILL = !KV8 ? 1 : SPLIT ? DW / 2 : DW;  // warps that fill a tile
    static constexpr int W_TMA = 4 * X, W_MMA = 4 * X + 1, W_CVT = 4 * X + 2;
    static constexpr int THREADS = 32 * (4 * X + 2 + DW);
    static constexpr int TMEM = 512;                 // two S of 128 columns, X O of T
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = X * TILE;
    static constexpr int OFF_V = OFF_K + KB * TILE;
    static constexpr int OFF_RAW = OFF_V + VB * TILE;
    static constexpr int OFF_SCALE = OFF_RAW + RU * RAW;
    // scale bytes of tiles whose rows do not share one: K[4], V[2]
    static constexpr int OFF_BYTES = OFF_SCALE + RU * kTile;
    static constexpr int OFF_RING = OFF_BYTES + (KV8 ? 6 * kTile : 0);  // [kRing] Seg
    static constexpr int OFF_BAR = OFF_RING + kRing * 48;
    // barriers
    static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + KB, B_VFULL = B_KEMPTY + KB,
                         B_VEMPTY = B_VFULL + VB, B_SFULL = B_VEMPTY + VB,
                         B_PFULL = B_SFULL + 2, B_O = B_PFULL + 2, B_LAND = B_O + 1,
                         B_POISON = B_LAND + 1, B_KFACT = B_POISON + kPoison, B_VFACT = B_KFACT + 4,
                         B_RFULL = B_VFACT + 2,
                         B_REMPTY = B_RFULL + RU, B_Q = B_REMPTY + RU, B_IFULL = B_Q + 1,
                         B_IEMPTY = B_IFULL + kRing, B_INFO = B_IEMPTY + kRing,
                         NBAR = B_INFO + kInfo;
    // tmem, abort, bad pages[kInfo] (8 bits each), poison[kPoison][4], scales: K[4], V[2]
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = 1024 + OFF_MISC + 112;
    static_assert(!KV8 || (KB <= 2 && VB <= 2), "f16 tiles");
    static_assert(VB <= kPoison && (kPoison & (kPoison - 1)) == 0, "poison words");
    static_assert(256 + X * T <= 512, "tensor memory");
    static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// What a request attends.  Lengths and offsets live on the device and are
// checked here: nothing outside [0, total_q) rows or the block table is used.
struct Req {
    int q_start, q_len, L;
    __device__ __forceinline__ int ctx() const { return max(L - q_len, 0); }
    // the first key any draft may see
    __device__ __forceinline__ int start(int window_left) const {
        return window_left < 0 ? 0 : max(ctx() - window_left, 0);
    }
};

__device__ __forceinline__ Req request(const TreeParams &p, int b, bool report) {
    Req r;
    const int a = p.cu_q[b], e = p.cu_q[b + 1], L = p.seqlens[b];
    bool bad = a < 0 || a > p.total_q;
    r.q_start = min(max(a, 0), p.total_q);
    long long n = (long long)e - a;
    if (n < 0 || n > p.max_seqlen_q || n > p.total_q - r.q_start) bad = true;
    n = n < 0 ? 0 : n;
    r.q_len = (int)min(n, (long long)min(p.max_seqlen_q, p.total_q - r.q_start));
    const long long cap_blocks = (long long)p.max_blocks_per_seq * p.block_size;
    const int cap = cap_blocks < p.max_seqlen ? (int)cap_blocks : p.max_seqlen;
    if (L < 0 || L > cap) bad = true;
    r.L = min(max(L, 0), cap);
    if (r.L < r.q_len) {  // the drafts are not all in the cache: nothing is attended
        bad = true;
        r.L = 0;
    }
    if (bad && report) flag_error(p.dev_error, PKV_DEVERR_SEQLEN);
    return r;
}

// A request on the line of work: its key tiles (one without keys, for the
// zeros), its row groups of `rows` rows, and their product.
struct Cost {
    int tiles, groups;
    __device__ __forceinline__ long long total() const { return (long long)tiles * groups; }
};

__device__ __forceinline__ Cost cost_of(const TreeParams &p, const Req &r, int rows) {
    Cost c;
    const int start = r.start(p.window_left);
    c.tiles = r.L > start ? (r.L - 1) / kTile - start / kTile + 1 : 1;
    c.groups = (r.q_len * p.group + rows - 1) / rows;
    return c;
}

// A segment: key tiles [tile0, tile0 + ntiles) of one row group of a request.
struct Seg {
    int q_start, q_len, ctx;
    int row0, nrows;               // the group's (draft, head) rows
    int tile0, ntiles;             // absolute key tiles; ntiles 0: no key at all
    int tok_lo, tok_hi;            // the keys of these tiles that are attended
    int full_lo, full_hi;          // tiles [full_lo, full_hi): every row sees every key
    int slot_b;                    // 4 * request + cut; -1: no more segments.  cut: 0 the
                                   // whole row group, 1 its begin is another CTA's (or both
                                   // ends are), 2 only its end is
    __device__ __forceinline__ int b() const { return slot_b >> 2; }
    __device__ __forceinline__ int cut() const { return slot_b & 3; }
    __device__ __forceinline__ bool partial(int j) const { return j < full_lo || j >= full_hi; }
};
static_assert(sizeof(Seg) == 48, "ring layout");

// The bounded wait of a whole warp (mbar_wait_bounded), written to be short: it
// stands at thirty places, and code that has to be fetched beside 150 streaming
// SMs takes microseconds.  It begins with a plain test, which costs a fraction of a
// try_wait where the phase is already complete (8 x 64 drafts 177 -> 173 us).
__device__ __noinline__ void gave_up(int32_t *dev_error, int32_t *abort) {
    flag_error(dev_error, PKV_DEVERR_TIMEOUT);
    if (abort) *reinterpret_cast<volatile int32_t *>(abort) = 1;
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, int32_t *dev_error,
                                         int32_t *abort = nullptr) {
    bool ok = mbar_test(bar, parity);
    if (!ok) {
        const long long t0 = clock64();
#pragma unroll 1
        while (!(ok = mbar_try_wait(bar, parity))) {
            if (abort && *reinterpret_cast<volatile int32_t *>(abort) != 0) break;
            if (clock64() - t0 > kWaitLimitCycles) {
                gave_up(dev_error, abort);
                break;
            }
        }
    }
    return ok;
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int32_t *dev_error,
                                          int32_t *abort = nullptr) {
    return __all_sync(0xffffffffu, wait_one(bar, parity, dev_error, abort));
}

// Bits n0 .. n0+31 of a draft's mask of nw 64-bit words (n0 may be negative).
__device__ __forceinline__ uint32_t mask_bits(const int64_t *m, int nw, int n0) {
    if (n0 <= -32 || n0 >= nw * 64) return 0u;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(m);
    if (n0 < 0) return w[0] << (-n0);
    const int i = n0 >> 5, s = n0 & 31;
    const uint32_t lo = w[i], hi = i + 1 < 2 * nw ? w[i + 1] : 0u;
    return __funnelshift_r(lo, hi, s);
}

// Bits [lo, hi) of a 32-bit word, for any lo and hi.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    if (lo >= hi) return 0u;
    const uint32_t top = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
    return top & ~((1u << lo) - 1u);
}

// ---------------------------------------------------------------------------
// Tiles over 8-bit pools whose rows do not share a scale: what the softmax does
// for them, key by key, on a warp's 32 rows of S at t_s.  Functions of their own,
// so that the usual tiles' code stays close together.
// ---------------------------------------------------------------------------
// Byte e of four words as a float less 127: 2^23 + byte has it in its last bits (a
// conversion would take the slow unit).
__device__ __forceinline__ float byte_exponent(const uint32_t (&b)[4], int e) {
    return __uint_as_float(__byte_perm(b[e / 4], 0x4b000000u, 0x7650 + e % 4)) - 8388735.f;
}

// S times f times 2^(its key's K exponent): the scores.
__device__ __noinline__ void scale_keys(uint32_t t_s, const uint8_t *bytes, float f) {
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t v[16];
        tc::ld_32x32b_x16(t_s + 16 * c, v);
        const uint4 b4 = *reinterpret_cast<const uint4 *>(bytes + 16 * c);
        const uint32_t b[4] = {b4.x, b4.y, b4.z, b4.w};
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
            v[e] = __float_as_uint(__uint_as_float(v[e]) * f *
                                   scale_value((b[e / 4] >> (8 * (e % 4))) & 255u));
        tc::st_32x32b_x16(t_s + 16 * c, v);
    }
    tc::wait_st();
}

// For weights by key: S becomes S * f + the exponent of its key's V scale (vexp for
// all keys without bytes).  Returns its largest, and the sum of 2^(S * f - top).
__device__ __noinline__ float2 add_exponents(uint32_t t_s, const uint8_t *bytes, float vexp,
                                             float f, float top) {
    float m = kNegInf, s0 = 0.f, s1 = 0.f;
    if (top == kNegInf) top = 0.f;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t v[16];
        tc::ld_32x32b_x16(t_s + 16 * c, v);
        uint4 b4 = make_uint4(0u, 0u, 0u, 0u);
        if (bytes) b4 = *reinterpret_cast<const uint4 *>(bytes + 16 * c);
        const uint32_t b[4] = {b4.x, b4.y, b4.z, b4.w};
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float x = __uint_as_float(v[e]);
            (e & 1 ? s1 : s0) += fast_exp2(fmaf(x, f, -top));
            const float y = fmaf(x, f, bytes ? byte_exponent(b, e) : vexp);
            m = fmaxf(m, y);
            v[e] = __float_as_uint(y);
        }
        tc::st_32x32b_x16(t_s + 16 * c, v);
    }
    tc::wait_st();
    return make_float2(m, s0 + s1);
}

template <int T, bool KV8, int X>
__global__ void __launch_bounds__(Cfg<T, KV8, X>::THREADS, 1)
tree_kernel(const TreeParams p, const __grid_constant__ CUtensorMap tmk,
            const __grid_constant__ CUtensorMap tmv) {
    using C = Cfg<T, KV8, X>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);  // 1024-aligned
    const uint32_t base = smem_u32(smem);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
    int32_t *s_abort = reinterpret_cast<int32_t *>(misc + 1);
    volatile uint8_t *s_bad = reinterpret_cast<uint8_t *>(misc + 2);  // [kInfo]
    uint32_t *s_poison = misc + 4;   // [kPoison][4]
    // K[4], V[2]: a tile's largest scale byte; 256 or more: its rows do not share one
    uint32_t *s_byte = misc + 4 + 4 * kPoison;
    Seg *ring = reinterpret_cast<Seg *>(smem + C::OFF_RING);
    auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };

    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = p.num_kv_heads, G = p.group, Dh = p.head_dim;
    const int g = blockIdx.x % Hkv, group = blockIdx.x / Hkv;
    const int BS = p.block_size, bs_shift = BS == 32 ? 5 : 4, npg = kTile >> bs_shift;

    // ---- set-up: barriers and TMEM
    if (threadIdx.x == 32 * C::W_TMA) {
        for (int i = 0; i < C::KB; ++i) {
            mbar_init(bar(C::B_KFULL + i), C::FILL);
            mbar_init(bar(C::B_KEMPTY + i), 1);
        }
        for (int i = 0; i < C::VB; ++i) {
            mbar_init(bar(C::B_VFULL + i), C::FILL);
            mbar_init(bar(C::B_VEMPTY + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::B_SFULL + i), 1);
            mbar_init(bar(C::B_PFULL + i), 4);
            mbar_init(bar(C::B_VFACT + i), 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(bar(C::B_KFACT + i), 1);
        for (int i = 0; i < kPoison; ++i) mbar_init(bar(C::B_POISON + i), C::FILL);
        mbar_init(bar(C::B_O), 1);
        mbar_init(bar(C::B_LAND), 1);
        mbar_init(bar(C::B_Q), 4 * X);
        for (int i = 0; i < C::RU; ++i) {
            mbar_init(bar(C::B_RFULL + i), 1 + 8);
            mbar_init(bar(C::B_REMPTY + i), C::FILL);
        }
        for (int i = 0; i < kInfo; ++i) mbar_init(bar(C::B_INFO + i), 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar(C::B_IFULL + i), 1);
            mbar_init(bar(C::B_IEMPTY + i), 4 * X + 1 + C::DW);
        }
        fence_barrier_init();
        *s_abort = 0;
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == C::W_MMA) {
        tc::tmem_alloc(base + C::OFF_MISC, C::TMEM);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    if (warp == C::W_TMA) {
        // the barriers are this warp's own work: it goes on, and only announces
        // that they are there
        __syncwarp();
        asm volatile("barrier.cta.arrive 1, %0;" ::"n"(C::THREADS) : "memory");
    } else {
        asm volatile("barrier.cta.sync 1, %0;" ::"n"(C::THREADS) : "memory");
    }
    tc::fence_after_sync();
    const uint32_t tmem = warp == C::W_TMA ? 0u : misc[0];

    // Segment n of this CTA lies in slot n % kRing of the ring, where the warps
    // read it until they release it; null: none left, or a wait gave up.
    auto segment = [&](int n) -> const Seg * {
        const int s = n % kRing;
        if (!wait_warp(bar(C::B_IFULL + s), (uint32_t)(n / kRing) & 1u, p.dev_error,
                               s_abort) ||
            ring[s].slot_b < 0)
            return nullptr;
        return ring + s;
    };
    auto release = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_IEMPTY + n % kRing));
    };

    if (warp == C::W_TMA) {
        // ------------------------------------------------------------ segments, loads
        constexpr int kRows = X * kTile;
        const int groups = gridDim.x / Hkv;
        // the line's length; the requests' places on it, and the share, go to the merge
        // kernel
        long long total = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            long long c = 0;
            if (b0 + lane < p.batch)
                c = cost_of(p, request(p, b0 + lane, blockIdx.x == 0), kRows).total();
            long long incl = c;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            if (blockIdx.x == 0 && b0 + lane < p.batch)
                p.line[b0 + lane] = total + incl - c;
            total += __shfl_sync(0xffffffffu, incl, 31);
        }
        const long long share =
            max((total + groups - 1) / groups, (long long)p.min_tiles);
        if (blockIdx.x == 0 && lane == 0) p.line[p.batch] = share;
        const long long lo = min(share * group, total), hi = min(lo + share, total);

        // box coordinates of (page, kv head); one past the pool reads zeros
        const int oob = p.hnd ? (int)(p.num_blocks * Hkv) : (int)(p.num_blocks * BS);
        const int cy = p.hnd ? 0 : g;
        bool alive = true;
        int nk = 0, nv = 0, nfix = 0;  // tiles (8-bit: raw tiles) and repaired tiles so far
        uint32_t landed = 0;           // bit i: the last use of V buffer i was a repaired tile
        // The boxes of a tile: page j's rows lie in lane j's `row`.
        auto load_tile = [&](const CUtensorMap *tm, uint32_t dst, uint32_t full, int row) {
            constexpr int B = KV8 ? C::ROWB : 128;           // bytes of a box row
            constexpr int PARTS = KV8 ? T / C::ROWB : C::HALVES;
            int rows[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) rows[j] = __shfl_sync(0xffffffffu, row, j);
            __syncwarp();
            if (elect_one()) {
                mbar_arrive_expect_tx(full, KV8 ? C::RAW : C::TILE);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < npg)
#pragma unroll
                        for (int h = 0; h < PARTS; ++h)
                            tma_load_3d(dst + h * (kTile * B) + j * BS * B, tm, full,
                                        h * (KV8 ? 128 : 64), cy, rows[j]);
            }
            __syncwarp();
        };
        auto load_segment = [&](const Seg &sg) {
            const int tok_lo = sg.tok_lo, tok_hi = sg.tok_hi;
            // 32 page ids per warp-wide load, a load ahead: beside 150 streaming SMs
            // it takes longer than a tile
            const int32_t *bt = p.block_table + (int64_t)sg.b() * p.max_blocks_per_seq;
            const int first = tok_lo >> bs_shift, last = (tok_hi - 1) >> bs_shift;
            const int tpb = 32 / npg;
            auto page_ids = [&](int i) {  // tiles i .. i + tpb - 1
                const int pg = (sg.tile0 + i) * npg + lane;
                return pg >= first && pg <= last ? bt[pg] : -1;
            };
            int ids = -1, ids_next = page_ids(0);
            // bf16: V goes one tile behind K, so that the products of the next tile's
            // K do not wait for the V slots
            int row_v = oob;
            for (int i = 0; i < sg.ntiles + (KV8 ? 0 : 1) && alive; ++i) {
                int row = oob, id = -1;
                if (KV8 || i < sg.ntiles) {
                    if (i % tpb == 0) {
                        ids = ids_next;
                        ids_next = page_ids(i + tpb);
                    }
                    id = __shfl_sync(0xffffffffu, ids, ((i % tpb) * npg + lane) & 31);
                    const int pg = (sg.tile0 + i) * npg + lane;
                    const bool attended = lane < npg && pg >= first && pg <= last;
                    const bool bad = attended && (id < 0 || id >= p.num_blocks);
                    if (bad) flag_error(p.dev_error, PKV_DEVERR_BLOCK_ID);
                    if (!attended || bad) id = -1;
                    if (id >= 0) row = p.hnd ? id * Hkv + g : id * BS;
                    const uint32_t badpg = __ballot_sync(0xffffffffu, bad);
                    const int jn = KV8 ? nk / 2 : nk;
                    if (lane == 0) {
                        s_bad[jn % kInfo] = (uint8_t)badpg;
                        mbar_arrive(bar(C::B_INFO + jn % kInfo));
                    }
                }
                if constexpr (!KV8) {
                    if (i < sg.ntiles) {
                        const int ks = nk % C::KB;
                        alive = wait_warp(bar(C::B_KEMPTY + ks),
                                          ((uint32_t)(nk / C::KB) & 1u) ^ 1u, p.dev_error,
                                          s_abort);
                        if (!alive) break;
                        load_tile(&tmk, base + C::OFF_K + ks * C::TILE, bar(C::B_KFULL + ks), row);
                        ++nk;
                    }
                    const int vrow = row_v;
                    row_v = row;
                    if (i == 0) continue;
                    const int iv = i - 1, vs = nv % C::VB;
                    alive = wait_warp(bar(C::B_VEMPTY + vs),
                                              ((uint32_t)(nv / C::VB) & 1u) ^ 1u, p.dev_error,
                                              s_abort);
                    if (!alive) break;
                    const bool fix = sg.partial(iv);
                    landed = fix ? landed | 1u << vs : landed & ~(1u << vs);
                    const uint32_t vbar = fix ? bar(C::B_LAND) : bar(C::B_VFULL + vs);
                    const uint32_t vb = base + C::OFF_V + vs * C::TILE;
                    load_tile(&tmv, vb, vbar, vrow);
                    ++nv;
                    if (fix) {
                        alive = wait_warp(bar(C::B_LAND), (uint32_t)nfix & 1u, p.dev_error,
                                                  s_abort);
                        ++nfix;
                        if (!alive) break;
                        // lane owns rows lane, lane + 32, ..: rows outside the range
                        // are zeroed, and rows with an infinity or a NaN, noted
                        uint32_t *pois = s_poison + ((nfix - 1) % kPoison) * 4;
                        const int k0 = (sg.tile0 + iv) * kTile;
#pragma unroll 1
                        for (int w = 0; w < 4; ++w) {
                            const int r = w * 32 + lane, key = k0 + r;
                            const bool in = key >= tok_lo && key < tok_hi;
                            bool bad = false;
                            if (in) {
#pragma unroll 4
                                for (int c = 0; c < T / 8; ++c) {
                                    const uint4 v =
                                        ld_shared16(vb + (c >> 3) * C::HALF + sw128(r, c & 7));
                                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        bad |= (x[e] & 0x7f80u) == 0x7f80u ||
                                               (x[e] & 0x7f800000u) == 0x7f800000u;
                                }
                            }
                            if (!in || bad)
                                for (int c = 0; c < T / 8; ++c)
                                    st_shared_zero16(vb + (c >> 3) * C::HALF + sw128(r, c & 7));
                            const uint32_t m = __ballot_sync(0xffffffffu, in && bad);
                            if (lane == 0) pois[w] = m;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(bar(C::B_POISON + (nfix - 1) % kPoison));
                            mbar_arrive(bar(C::B_VFULL + vs));
                        }
                    }
                } else {
                    // scale bytes: lane l < 8 copies bytes 16 l .. of the tile
                    const int sid = __shfl_sync(0xffffffffu, id, (lane * 16 >> bs_shift) & 31);
                    for (int v = 0; v < 2 && alive; ++v) {
                        const int s = nk % C::RU;
                        const uint32_t full = bar(C::B_RFULL + s);
                        alive = wait_warp(bar(C::B_REMPTY + s),
                                                  ((uint32_t)(nk / C::RU) & 1u) ^ 1u, p.dev_error,
                                                  s_abort);
                        if (!alive) break;
                        load_tile(v ? &tmv : &tmk, base + C::OFF_RAW + s * C::RAW, full, row);
                        if (lane < 8) {
                            if (sid >= 0)
                                cp_async16(base + C::OFF_SCALE + s * kTile + lane * 16,
                                           (v ? p.v_scale : p.k_scale) +
                                               ((int64_t)sid * Hkv + g) * BS +
                                               (lane * 16) % BS);
                            cp_async_arrive(full);
                        }
                        ++nk;
                    }
                }
            }
            return alive;
        };
        int nseg = 0;
        long long place = 0;           // where the chunk's first request begins
        for (int b0 = 0; b0 < p.batch && place < hi && alive; b0 += 32) {
            Req mine = {0, 0, 0};
            long long c = 0;
            if (b0 + lane < p.batch) {
                mine = request(p, b0 + lane, false);
                c = cost_of(p, mine, kRows).total();
            }
            long long incl = c;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            const long long first = place + incl - c;
            place += __shfl_sync(0xffffffffu, incl, 31);
            // the requests of this chunk that meet [lo, hi)
            uint32_t meet = __ballot_sync(0xffffffffu, c > 0 && first < hi && first + c > lo);
            for (; meet && alive; meet &= meet - 1) {
                const int src = __ffs(meet) - 1;
                Req rq;
                rq.q_start = __shfl_sync(0xffffffffu, mine.q_start, src);
                rq.q_len = __shfl_sync(0xffffffffu, mine.q_len, src);
                rq.L = __shfl_sync(0xffffffffu, mine.L, src);
                const long long at = __shfl_sync(0xffffffffu, first, src);
                const Cost co = cost_of(p, rq, kRows);
                const int start = rq.start(p.window_left);
                int wfull = 0;
                if (p.window_left >= 0) {  // the deepest draft bounds what all rows see
                    int d = 0;
                    for (int i = lane; i < rq.q_len; i += 32) d = max(d, p.depth[rq.q_start + i]);
                    d = __reduce_max_sync(0xffffffffu, d);
                    wfull = (int)min(max((long long)rq.ctx() + d - p.window_left, 0LL),
                                     (long long)rq.L);
                }
                for (int rg = 0; rg < co.groups && alive; ++rg) {
                    const long long s = at + (long long)rg * co.tiles, e = s + co.tiles;
                    if (e <= lo || s >= hi) continue;
                    const int t0 = (int)(max(s, lo) - s), t1 = (int)(min(e, hi) - s);
                    Seg sg;
                    sg.q_start = rq.q_start;
                    sg.q_len = rq.q_len;
                    sg.ctx = rq.ctx();
                    sg.row0 = rg * kRows;
                    sg.nrows = min(rq.q_len * G - sg.row0, kRows);
                    sg.tile0 = start / kTile + t0;
                    sg.ntiles = rq.L > start ? t1 - t0 : 0;
                    sg.tok_lo = max(sg.tile0 * kTile, start);
                    sg.tok_hi =
                        (int)min((long long)(sg.tile0 + sg.ntiles) * kTile, (long long)rq.L);
                    sg.full_lo = (max(sg.tok_lo, wfull) + kTile - 1) / kTile - sg.tile0;
                    sg.full_hi = min(sg.tok_hi, sg.ctx) / kTile - sg.tile0;
                    sg.slot_b = 4 * (b0 + src) + (lo > s ? 1 : hi < e ? 2 : 0);
                    const int rs = nseg % kRing;
                    alive = wait_warp(bar(C::B_IEMPTY + rs),
                                              ((uint32_t)(nseg / kRing) & 1u) ^ 1u, p.dev_error,
                                              s_abort);
                    if (!alive) break;
                    if (lane == 0) {
                        ring[rs] = sg;
                        mbar_arrive(bar(C::B_IFULL + rs));
                    }
                    ++nseg;
                    if (sg.ntiles > 0) alive = load_segment(sg);
                }
            }
        }
        if (alive) {  // no more
            const int rs = nseg % kRing;
            alive = wait_warp(bar(C::B_IEMPTY + rs),
                                      ((uint32_t)(nseg / kRing) & 1u) ^ 1u, p.dev_error, s_abort);
            if (alive && lane == 0) {
                ring[rs].slot_b = -1;
                mbar_arrive(bar(C::B_IFULL + rs));
            }
        }
        if (!alive) {  // a wait gave up: let the copies in flight land (bounded)
            if constexpr (!KV8) {
                for (int i = max(0, nk - C::KB); i < nk; ++i)
                    wait_warp(bar(C::B_KFULL + i % C::KB), (uint32_t)(i / C::KB) & 1u,
                                      p.dev_error);
                for (int i = max(0, nv - C::VB); i < nv; ++i)
                    if (!((landed >> (i % C::VB)) & 1u))
                        wait_warp(bar(C::B_VFULL + i % C::VB),
                                          (uint32_t)(i / C::VB) & 1u, p.dev_error);
                if (nfix > 0)
                    wait_warp(bar(C::B_LAND), (uint32_t)(nfix - 1) & 1u, p.dev_error);
            } else {
                for (int u = max(0, nk - C::RU); u < nk; ++u)
                    wait_warp(bar(C::B_RFULL + u % C::RU), (uint32_t)(u / C::RU) & 1u,
                                      p.dev_error);
            }
        }
    } else if (warp == C::W_MMA) {
        // ------------------------------------------------------------ MMA issuer
        // f16 operands over 8-bit pools, bf16 otherwise (A and B alike; the
        // format fields are bits 7 and 10)
        constexpr uint32_t fmt = KV8 ? (1u << 7 | 1u << 10) : 0u;
        constexpr uint32_t idS = tc::idesc_bf16_f32(128, 128, 0, 0) & ~fmt;
        constexpr uint32_t idO = tc::idesc_bf16_f32(128, T, 0, 1) & ~fmt;
        const uint64_t dq0 = tc::smem_desc_sw128(base + C::OFF_Q, 16, 1024);
        const uint64_t dk0 = tc::smem_desc_sw128(base + C::OFF_K, 16, 1024);
        const uint64_t dv0 = tc::smem_desc_sw128(base + C::OFF_V, C::HALF, 1024);
        // One thread issues, and spends as little as it can between two products:
        // the tensor pipe runs dry meanwhile (buffer indexes and phases are
        // counted, not divided out).
        auto wait = [&](int i, uint32_t phase) {
            return wait_one(bar(i), phase, p.dev_error, s_abort);
        };
        int ks = 0, vs = 0;             // K buffer of the next S, V buffer of the next O
        uint32_t kph = 0, vph = 0;      // and their phases
        int un = 0;                     // units so far
        bool alive = true;
        for (int ns = 0; alive; ++ns) {
            const Seg *sg = segment(ns);
            if (!sg) break;
            const int nx = sg->nrows > kTile ? 2 : 1, total = sg->ntiles * nx;
            release(ns);
            if (elect_one()) {
                int sx = 0;             // row tile of the next S
                bool k_ready = false;
                // S of unit n; `must`: waits for its K tile, else gives up if that is
                // not there.  Returns 1 when issued, 0 when not, -1 when a wait gave up.
                auto issue_s = [&](int n, bool must) {
                    if (!k_ready) {
                        if (must) {
                            if (!wait(C::B_KFULL + ks, kph)) return -1;
                        } else if (!mbar_test(bar(C::B_KFULL + ks), kph)) {
                            return 0;
                        }
                    }
                    k_ready = true;
                    tc::fence_after_sync();
                    const uint64_t dq = dq0 + (uint64_t)((sx * C::TILE) >> 4);
                    const uint64_t dk = dk0 + (uint64_t)((ks * C::TILE) >> 4);
                    const uint32_t d = tmem + (n & 1) * 128;
                    if constexpr (T == 128) {
                        tc::mma_ss8<C::HALF>(d, dq, dk, idS, 0u);
                    } else {
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t off = (h * C::HALF + k * 32) >> 4;
                                tc::mma_ss(d, dq + off, dk + off, idS, h + k > 0 ? 1u : 0u);
                            }
                    }
                    tc::commit(bar(C::B_SFULL + (n & 1)));
                    if (++sx == nx) {
                        tc::commit(bar(C::B_KEMPTY + ks));
                        sx = 0;
                        k_ready = false;
                        if (++ks == C::KB) {
                            ks = 0;
                            kph ^= 1u;
                        }
                    }
                    return 1;
                };
                alive = wait(C::B_Q, (uint32_t)ns & 1u);
                int x = 0, issued = 0;  // row tile of the next O; S so far
                for (int i = 0; i < total && alive; ++i) {
                    // S runs up to two units ahead of O, but does not hold O up when
                    // its K tile is late
                    while (issued < total && issued < i + 2) {
                        const int did = issue_s(un + issued, issued == i);
                        alive = did >= 0;
                        if (did <= 0) break;
                        ++issued;
                    }
                    if (!alive) break;
                    const int n = un + i;
                    alive = wait(C::B_PFULL + (n & 1), (uint32_t)(n >> 1) & 1u) &&
                            (x > 0 || wait(C::B_VFULL + vs, vph));
                    if (!alive) break;
                    tc::fence_after_sync();
                    const uint64_t dv = dv0 + (uint64_t)((vs * C::TILE) >> 4);
                    tc::mma_ts8(tmem + 256 + x * T, tmem + (n & 1) * 128, dv, idO,
                                i >= nx ? 1u : 0u);
                    if (++x == nx) {
                        tc::commit(bar(C::B_VEMPTY + vs));
                        x = 0;
                        if (++vs == C::VB) {
                            vs = 0;
                            vph ^= 1u;
                        }
                    }
                }
                tc::commit(bar(C::B_O));  // (with nothing in flight it arrives at once)
                un += total;
                // a wait gave up: let the products in flight finish (bounded)
                if (!alive) wait_one(bar(C::B_O), (uint32_t)ns & 1u, p.dev_error);
            }
            alive = __all_sync(0xffffffffu, alive);
        }
        __syncwarp();
    } else if (warp < 4 * X) {
        // ------------------------------------------------------------ softmax
        const int x = warp >> 2;             // row tile
        const int r = threadIdx.x;           // row of the CTA; TMEM lane r % 128
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_o = tmem + 256 + x * T + lane_base;
        const uint32_t sq = base + C::OFF_Q + x * C::TILE;
        // (draft, head) of this thread's row, as its index in q, out and lse
        auto unit_of = [&](const Seg &sg) {
            const int i = sg.row0 + min(r, sg.nrows - 1), tok = i / G;
            return (int64_t)(sg.q_start + tok) * p.num_qo_heads + g * G + (i - tok * G);
        };
        const bool positions = p.window_left >= 0 || p.alibi;
        uint32_t un = 0, jt = 0, nfix = 0;   // units, key tiles and repaired tiles so far
        bool alive = true;
        // Segment by segment: Q on its way, the rows of the segment before stored
        // meanwhile, Q's last touch, the key tiles.
        const Seg *prev = nullptr;
        float m_ref = kNegInf, l_ref = kNegInf, l = 0.f, sink = kNegInf;
        bool poisoned = false;               // the row keeps a key whose V is not finite
        int64_t unit = 0;
#pragma unroll 1
        for (int ns = 0;; ++ns) {
        const Seg *sp = segment(ns);         // stays in the ring until it is released
        const int64_t unit_prev = unit;
        if (sp) {
            // this warp's rows of Q into shared memory (rows past the last: zeros),
            // LPR lanes per row
            unit = unit_of(*sp);
            constexpr int LPR = T / 8 < 32 ? T / 8 : 32, RPS = 32 / LPR;
            const int c = lane % LPR, r0 = lane / LPR, nrows = sp->nrows;
            const bool col_on = c * 8 < Dh;
            // the lane's first row as (draft, head of the group); RPS rows on, the
            // head moves by RPS % G, and the draft by RPS / G or one more
            const int i0 = sp->row0 + warp * 32 + r0, tok0 = i0 / G;
            int rem = i0 - tok0 * G;
            const int dr = RPS % G;
            const int64_t Hq = p.num_qo_heads, step = (RPS / G) * Hq + dr;
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) + c * 8 +
                                       ((sp->q_start + tok0) * Hq + g * G + rem) * Dh;
#pragma unroll 2
            for (int k = 0; k < 32 / RPS; ++k) {
                const int rr = k * RPS + r0, row = (warp & 3) * 32 + rr;
                const bool on = col_on && warp * 32 + rr < nrows;
                cp_async16_or_zero(sq + (c >> 3) * C::HALF + sw128(row, c & 7), on ? src : p.q, on);
                src += step * Dh;
                rem += dr;
                if (rem >= G) {
                    rem -= G;
                    src += (Hq - G) * Dh;
                }
            }
            // the row's mask, read in the last key tiles
            if (r < nrows)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(
                    p.mask + (int64_t)(sp->q_start + (sp->row0 + r) / G) * p.mask_words));
        }
        if (prev && prev->nrows > warp * 32) {
            // ---- the rows' results
            const Seg &sg = *prev;
            tc::fence_after_sync();
            // partials: [CTA group][its first or last row group][kv head], there lse
            // [row] and O [D / 4][row][4], so that the rows' threads store whole lines
            // (row by row, 3900 cycles of stores instead of 1000)
            const bool part = sg.cut() != 0, row_on = r < sg.nrows;
            const int64_t pslot = (int64_t)(2 * group + sg.cut() / 2) * Hkv + g;
            float4 *po = reinterpret_cast<float4 *>(p.part_o) + pslot * (Dh / 4) * (X * kTile) + r;
            float mul, lse, h = 1.f;
            if (!KV8)
                l_ref = m_ref;
            else  // O's units, 2^(m_ref - l_ref), in two halves: the whole may overflow
                h = l_ref == kNegInf ? 0.f : exp2f(0.5f * (m_ref - l_ref));
            if (part) {
                mul = l == 0.f ? 0.f : 1.f / l;
                lse = l == 0.f ? kNegInf : l_ref + log2f(l);
                if (row_on) p.part_lse[pslot * (X * kTile) + r] = lse;
            } else {
                const float M = fmaxf(l_ref, sink);
                const float Ms = M == kNegInf ? 0.f : M;
                const float f = exp2f(l_ref - Ms);
                const float lam = l * f + exp2f(sink - Ms);
                mul = lam == 0.f ? 0.f : f / lam;
                lse = lam == 0.f ? kNegInf : (Ms + log2f(lam)) * kLn2;
                // a NaN weight leaves the reference as it was: keep the NaN
                if (l != l) mul = lse = l;
                if (row_on && p.lse_out) p.lse_out[unit_prev] = lse;
            }
            // (its V row was zeroed; the lse is of the scores alone)
            if (poisoned) mul = __uint_as_float(0x7fffffffu);
            // Each thread stores its row, 16 columns at a time: whole sectors, without
            // a turn through shared memory, where the next segment's Q is landing.
#pragma unroll 1
            for (int c = 0; c < T / 16; ++c) {
                uint32_t v[16];
                tc::ld_32x32b_x16(t_o + 16 * c, v);
                tc::wait_ld();
                float o[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = sg.ntiles == 0 ? 0.f
                           : KV8          ? __uint_as_float(v[e]) * mul * h * h
                                          : __uint_as_float(v[e]) * mul;
                const bool on = row_on && 16 * c < Dh;
                if (on && part) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        po[(4 * c + e) * (X * kTile)] =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else if (on) {
                    uint4 *at = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                                          unit_prev * Dh + 16 * c);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        at[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]),
                                           pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                           pack_bf16(o[8 * e + 4], o[8 * e + 5]),
                                           pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                }
                __syncwarp();
            }
            tc::fence_before_sync();
        }
        if (prev) release(ns - 1);
        if (!sp) break;
        const Seg &sg = *sp;
        prev = sp;
        const int ntiles = sg.ntiles, nx = sg.nrows > kTile ? 2 : 1;
        const int full_lo = sg.full_lo, full_hi = sg.full_hi;
        const bool warp_on = warp * 32 < sg.nrows, row_on = r < sg.nrows;
        float rowf = fabsf(p.scale_log2);    // score = S * rowf
        {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            const uint32_t neg = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // its sign goes into q
            if (KV8 || neg) {
                // this thread's row in place: to f16, times a power of two that brings
                // its largest value to 2^14..2^15 (exact down to 2^-28 of it)
                const uint32_t row = (uint32_t)r % kTile;
                uint32_t m = 0;
                float f = 1.f;
                if constexpr (KV8) {
#pragma unroll 4
                    for (int k = 0; k < T / 8; ++k) {
                        const uint4 v = ld_shared16(sq + (k >> 3) * C::HALF + sw128(row, k & 7));
                        m = bf16x2_max_nan(m, bf16x2_max_nan(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu));
                        m = bf16x2_max_nan(m, bf16x2_max_nan(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                    }
                    const int E = max((int)(max(m & 0xffffu, m >> 16) >> 7) - 127, -100);
                    f = __uint_as_float((uint32_t)(127 + 14 - E) << 23);
                    rowf *= __uint_as_float((uint32_t)(127 + E - 14) << 23);
                }
#pragma unroll 2
                for (int k = 0; k < T / 8; ++k) {
                    const uint32_t at = sq + (k >> 3) * C::HALF + sw128(row, k & 7);
                    const uint4 v = ld_shared16(at);
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (KV8)
                            w[e] = pack_f16(__uint_as_float(w[e] << 16) * f,
                                            __uint_as_float(w[e] & 0xffff0000u) * f);
                        w[e] ^= neg;
                    }
                    st_shared16(at, w[0], w[1], w[2], w[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_Q));
        }
        // Weights are 2^(s - m_ref), and m_ref follows the row's largest score.  Over
        // 8-bit pools they are 2^(s + v - m_ref) with the exponent v of the tile's
        // (or the key's) V scale, and m_ref follows the largest s + v, less kWeightExp,
        // so that f16 holds them; the sum l is there of 2^(s - l_ref).
        m_ref = l_ref = kNegInf;
        l = 0.f;
        poisoned = false;
        for (int j = 0; j < ntiles && x < nx; ++j) {
            const uint32_t n = un + j * nx + x, jn = jt + j;
            const uint32_t t_s = tmem + (n & 1) * 128 + lane_base;
            const bool fix = j < full_lo || j >= full_hi;
            alive = wait_warp(bar(C::B_INFO + jn % kInfo), (jn / kInfo) & 1u, p.dev_error,
                              s_abort);
            // the scales, on their way before S is there (heads of 64: 121 us instead of 118
            // for 8 x 32 drafts over 16K..24K when V's is waited for where it is used)
            uint32_t kb = 0, vb = 0;
            if constexpr (KV8) {
                alive = alive &&
                        wait_warp(bar(C::B_KFACT + (jn & 3)), (jn >> 2) & 1u, p.dev_error,
                                  s_abort) &&
                        wait_warp(bar(C::B_VFACT + (jn & 1)), (jn >> 1) & 1u, p.dev_error,
                                  s_abort);
                kb = *reinterpret_cast<volatile uint32_t *>(s_byte + (jn & 3));
                vb = *reinterpret_cast<volatile uint32_t *>(s_byte + 4 + (jn & 1));
            }
            alive = alive && wait_warp(bar(C::B_SFULL + (n & 1)), (n >> 1) & 1u, p.dev_error,
                                       s_abort);
            if (fix && alive) {
                alive = wait_warp(bar(C::B_POISON + nfix % kPoison), (nfix / kPoison) & 1u,
                                  p.dev_error, s_abort);
                ++nfix;
            }
            const uint32_t badpg = s_bad[jn % kInfo];
            if (!alive) break;
            if (warp_on) {
                tc::fence_after_sync();
                float rf = rowf;
                if constexpr (KV8) rf *= kb > 255u ? 1.f : scale_value(kb);
                const bool general = fix || badpg != 0 || p.alibi != nullptr || kb > 255u;
                // General tiles.  The keys among kc .. kc + 31 that draft `node` at position
                // qpos sees.
                auto depth_of = [&](int k) {  // a draft's depth
                    return positions ? min(max(p.depth[sg.q_start + k], 0), 65535) : 0;
                };
                auto visible = [&](int kc, int node, int qpos) {
                    const int ctx = sg.ctx, tok_lo = sg.tok_lo, tok_hi = sg.tok_hi;
                    const int wlo = p.window_left < 0 ? 0 : max(qpos - p.window_left, 0);
                    uint32_t vis = range_bits(max(wlo, tok_lo) - kc, min(ctx, tok_hi) - kc);
                    const int n0 = kc - ctx;  // draft node of the first key
                    if (n0 > -32 && n0 < sg.q_len && row_on) {
                        uint32_t d =
                            mask_bits(p.mask + (int64_t)(sg.q_start + node) * p.mask_words,
                                      p.mask_words, n0);
                        d &= range_bits(max(tok_lo, ctx) - kc, tok_hi - kc);
                        if (p.window_left >= 0) {
                            for (uint32_t m = d; m; m &= m - 1) {
                                const int e = __ffs(m) - 1;
                                if (ctx + depth_of(n0 + e) < qpos - p.window_left)
                                    d &= ~(1u << e);
                            }
                        }
                        vis |= d;
                    }
                    return vis;
                };
                // Chunk c (16 keys) of S as complete scores in log2 units: with bias,
                // -inf for what the row does not see.  A key that it sees and whose V row
                // is not finite poisons the row.  Short, because it is mostly fetched for
                // one tile.
                auto complete = [&](int c, uint32_t vis, int head, int qpos, uint32_t (&v)[16]) {
                    if ((badpg >> (c * 16 >> bs_shift)) & 1u) vis = 0u;
                    const uint32_t pois =
                        fix ? *reinterpret_cast<volatile uint32_t *>(
                                  s_poison + ((nfix - 1) % kPoison) * 4 + (c >> 1)) >>
                                  (c & 1) * 16
                            : 0u;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] = __float_as_uint(__uint_as_float(v[e]) * rf);
                    if (p.alibi) {
                        // lane e holds the position of the chunk's key e
                        const float slope = p.alibi[g * G + head] * kLog2e;
                        const int ctx = sg.ctx;
                        const int k = (sg.tile0 + j) * kTile + 16 * c + lane;
                        const int kpos =
                            k < ctx ? k : ctx + depth_of(min(k - ctx, sg.q_len - 1));
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[e] = __float_as_uint(
                                fmaf(slope, (float)(__shfl_sync(0xffffffffu, kpos, e) - qpos),
                                     __uint_as_float(v[e])));
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (!((vis >> e) & 1u)) v[e] = __float_as_uint(kNegInf);
                    poisoned |= (pois & vis & 0xffffu) != 0u;
                };
                auto maximum = [&](float m, const auto &v) {
                    float a0 = m, a1 = kNegInf;
#pragma unroll
                    for (int e = 0; e < (int)(sizeof v / 4); e += 4) {
                        a0 = fmax3(a0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                        a1 = fmax3(a1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                    }
                    return fmaxf(a0, a1);
                };
                // Weights of chunk c, 2^(v * f - m): their sum, and 16 columns of P
                // over S columns that have been read.
                auto weights = [&](int c, const uint32_t (&v)[32], float f, float m) {
                    float s0 = 0.f, s1 = 0.f;
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float a = fast_exp2(fmaf(__uint_as_float(v[e]), f, -m));
                        const float b = fast_exp2(fmaf(__uint_as_float(v[e + 1]), f, -m));
                        s0 += a;
                        s1 += b;
                        w[e / 2] = KV8 ? pack_f16(a, b) : pack_bf16(a, b);
                    }
                    tc::st_32x32b_x16(t_s + 16 * c, w);
                    return s0 + s1;
                };
                // The row's references move up to sm, its largest score, and to mt, its
                // largest weight's exponent; returns false if a wait gave up.
                auto refer = [&](float sm, float mt) {
                    if (KV8 && sm > l_ref + kLazySum) {
                        l *= fast_exp2(l_ref - sm);
                        l_ref = sm;
                    }
                    const bool grow = mt > m_ref + kLazy<KV8>;  // (-inf: by anything)
                    if (KV8 && !__any_sync(0xffffffffu, grow)) return true;
                    if (nx == 1) {  // O must be at rest: the last PV is done
                        // (with two row tiles, S(n) came behind this O's last PV)
                        if (!wait_warp(bar(C::B_VEMPTY + (jn - 1) % C::VB),
                                               (uint32_t)((jn - 1) / C::VB) & 1u, p.dev_error,
                                               s_abort))
                            return false;
                        tc::fence_after_sync();
                    }
                    const float f = grow ? fast_exp2(m_ref - mt) : 1.f;
                    if (grow) m_ref = mt;
                    if (!KV8) l *= f;
#pragma unroll 1
                    for (int c = 0; c < T / 16; ++c) {
                        uint32_t o[16];
                        tc::ld_32x32b_x16(t_o + 16 * c, o);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc::st_32x32b_x16(t_o + 16 * c, o);
                    }
                    return true;
                };
                // Twice over S, in loops: unrolled over the row, the code alone outgrows
                // the schedulers' instruction caches (the second pass by 64 keys at a time
                // instead of 32: 151 -> 160 us for 8 x 32 drafts over 24K of 8-bit).  The
                // first pass takes the maximum, and in a general tile leaves the completed
                // scores behind.
                float mt = kNegInf;
                if (!general) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[2][32];
                        tc::ld_32x32b_x32(t_s + 64 * h, v[0]);
                        tc::ld_32x32b_x32(t_s + 64 * h + 32, v[1]);
                        tc::wait_ld();
                        mt = maximum(maximum(mt, v[0]), v[1]);
                    }
                } else {
                    const int i = sg.row0 + min(r, sg.nrows - 1), node = i / G;
                    const int qpos = sg.ctx + depth_of(node);
                    uint32_t vis = 0u;
                    if (KV8 && kb > 255u) {
                        scale_keys(t_s, smem + C::OFF_BYTES + (jn & 3) * kTile, rf);
                        rf = 1.f;
                    }
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        vis = c & 1 ? vis >> 16
                                    : visible((sg.tile0 + j) * kTile + 16 * c, node, qpos);
                        __syncwarp();
                        uint32_t v[16];
                        tc::ld_32x32b_x16(t_s + 16 * c, v);
                        tc::wait_ld();
                        complete(c, vis, i - node * G, qpos, v);
                        __syncwarp();
                        mt = maximum(mt, v);
                        tc::st_32x32b_x16(t_s + 16 * c, v);
                    }
                    tc::wait_st();
                    rf = 1.f;
                }
                mt *= rf;
                float wt = mt, vexp = 0.f;  // the largest weight's exponent; V's scale in it
                bool by_key = false;
                if constexpr (KV8) {
                    vexp = (float)((int)(vb & 255u) - 127);
                    wt = mt + vexp - kWeightExp;
                    by_key = vb > 255u;
                }
                // The sum over 8-bit pools is that of the weights, moved by m_ref - vexp -
                // l_ref, unless V's scales differ from key to key, or are so far below those
                // that m_ref stands for that what counts in it would underflow as a weight.
                auto far = [&] { return KV8 && m_ref - vexp - l_ref > kLazySum; };
                if (j == 0 && !by_key) {
                    m_ref = wt;
                    l_ref = mt;
                } else if (by_key ||
                           __any_sync(0xffffffffu, wt > m_ref + kLazy<KV8> ||
                                                       (KV8 && mt > l_ref + kLazySum) || far())) {
                    float key_sum = 0.f;
                    if constexpr (KV8) {
                        const bool bytes = by_key;
                        by_key = by_key || __any_sync(0xffffffffu, far());
                        if (by_key) {
                            const float2 of = add_exponents(
                                t_s, bytes ? smem + C::OFF_BYTES + (4 + (jn & 1)) * kTile : nullptr,
                                vexp, rf, mt);
                            wt = of.x - kWeightExp;
                            key_sum = of.y;
                            rf = 1.f;
                            vexp = 0.f;
                        }
                    }
                    if (j == 0) {
                        m_ref = wt;
                        l_ref = mt;
                    } else {
                        alive = refer(mt, wt);
                        if (!alive) break;
                    }
                    if (by_key && mt != kNegInf) l += key_sum * fast_exp2(mt - l_ref);
                }
                const float m = (m_ref == kNegInf ? 0.f : m_ref) - vexp;
                float sum = 0.f;
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {
                    uint32_t v[32];
                    tc::ld_32x32b_x32(t_s + 32 * h, v);
                    tc::wait_ld();
                    sum += weights(h, v, rf, m);
                }
                if (KV8)
                    sum *= by_key ? 0.f
                                  : fast_exp2(fminf(m - (l_ref == kNegInf ? 0.f : l_ref), kLazySum));
                l += sum;
                tc::wait_st();
                tc::fence_before_sync();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_PFULL + (n & 1)));
        }
        un += ntiles * nx;
        jt += ntiles;
        if (x >= nx)  // this row tile is empty: its repaired tiles count all the same
            nfix += ntiles - max(min(full_hi, ntiles) - max(full_lo, 0), 0);
        sink = p.sink && row_on ? p.sink[g * G + (sg.row0 + r) % G] * kLog2e : kNegInf;
        // every product of the segment is done: O is at rest and Q's tile free
        if (alive)
            alive = wait_warp(bar(C::B_O), (uint32_t)ns & 1u, p.dev_error, s_abort);
        if (!alive) break;
        }
    } else if constexpr (KV8) {
        // ------------------------------------------------------------ codes -> f16 tiles
        // 128 / DW rows of every K and V tile per warp; a lane converts 16 codes at
        // a time.  Rows r and r ^ 5 go side by side: their 16-byte chunks, four of
        // each, meet no bank twice, neither where they are read nor written.
        constexpr int ROWS = kTile / C::FILL;
        const int w = (warp - C::W_CVT) % C::FILL, side = (warp - C::W_CVT) / C::FILL;
        bool alive = true;
        uint32_t jt = 0, nfix = 0;           // key tiles and repaired tiles so far
        for (int ns = 0; alive; ++ns) {
        const Seg *sp = segment(ns);
        if (!sp) break;
        const Seg &sg = *sp;                 // stays in the ring until it is released
        const int tok_lo = sg.tok_lo, tok_hi = sg.tok_hi;
        for (int i = 0; i < sg.ntiles && alive; ++i, ++jt) {
            const int k0 = (sg.tile0 + i) * kTile;
            uint32_t in4 = 0;  // lane: which of rows 4 lane .. 4 lane + 3 are attended
            const bool fix = sg.partial(i);
#pragma unroll 1
            for (int isv = side; isv < (C::SPLIT ? side + 1 : 2); ++isv) {
                const uint32_t u = 2 * jt + isv, rs = u % C::RU;
                const uint32_t nb = isv ? C::VB : C::KB, s = nb == 1 ? 0u : jt % 2;
                const uint32_t turn = nb == 1 ? jt : jt / 2;
                alive = wait_warp(bar(C::B_RFULL + rs), (uint32_t)(u / C::RU) & 1u,
                                          p.dev_error, s_abort) &&
                        wait_warp(bar((isv ? C::B_VEMPTY : C::B_KEMPTY) + s),
                                          (turn & 1u) ^ 1u, p.dev_error, s_abort);
                if (!alive) break;
                in4 = 0;
                if (!((s_bad[jt % kInfo] >> (lane * 4 >> bs_shift)) & 1u))
                    in4 = range_bits(tok_lo - k0 - 4 * lane, tok_hi - k0 - 4 * lane) & 15u;
                const uint8_t *sc = smem + C::OFF_SCALE + rs * kTile;
                // Row r = 8 * group + rq: its chunks' places in the raw tile and in the
                // f16 tile depend on the group only through 8 rows' distance.
                const int q = lane >> 3, c4 = lane & 3, rq = (lane & 4) ? q ^ 5 : q;
                const uint8_t *src = smem + C::OFF_RAW + rs * C::RAW + w * ROWS * C::ROWB;
                uint8_t *dst = smem + (isv ? C::OFF_V : C::OFF_K) + s * C::TILE + w * ROWS * 128;
                uint32_t so[C::HALVES];
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h) {
                    const int c = h * 4 + c4, part_c = (c * 16) / C::ROWB;
                    const int cc = c - part_c * (C::ROWB / 16);
                    so[h] = part_c * (kTile * C::ROWB) +
                            (C::ROWB == 128 ? sw128(rq, cc)
                                            : rq * 64u + ((cc ^ ((rq >> 1) & 3)) << 4));
                }
                const uint32_t do0 = sw128(rq, 2 * c4), do1 = sw128(rq, 2 * c4 + 1);
                // This lane's four bytes at once.  attended: a byte of ones per row; nan:
                // the top bit of a NaN row's
                const uint32_t b4 = *reinterpret_cast<const uint32_t *>(sc + 4 * lane);
                const uint32_t attended = (in4 * 0x00204081u & 0x01010101u) * 255u;
                const uint32_t x4 = b4 & attended;
                const uint32_t nan = x4 & ((x4 & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                // the largest and the smallest scale of the attended rows, NaN rows aside
                const uint32_t hi4 = x4 & ~((nan >> 7) * 255u), lo4 = b4 | ~attended;
                const uint32_t hi2 = __vmaxu2(hi4 & 0x00ff00ffu, (hi4 >> 8) & 0x00ff00ffu);
                const uint32_t lo2 = __vminu2(lo4 & 0x00ff00ffu, (lo4 >> 8) & 0x00ff00ffu);
                const uint32_t top = __reduce_max_sync(0xffffffffu, max(hi2 & 0xffffu, hi2 >> 16));
                const bool wide = __any_sync(
                    0xffffffffu, min(lo2 & 0xffffu, lo2 >> 16) + (isv ? kSpreadV : kSpreadK) < top);
                if (w == 0) {
                    // The softmax that last used the slot is done: V's that of two tiles
                    // ago, as its buffer is free; K's that of four tiles ago, as S of
                    // two tiles ago is done, which came behind that tile's O.
                    const int slot = isv ? 4 + (jt & 1) : jt & 3;
                    if (wide)  // (a NaN row's values are NaN whatever its scale: 0, which
                               // counts for no maximum)
                        *reinterpret_cast<uint32_t *>(smem + C::OFF_BYTES + slot * kTile +
                                                      4 * lane) = b4 & ~((nan >> 7) * 255u);
                    __syncwarp();
                    if (lane == 0) {
                        s_byte[slot] = top | (wide ? 256u : 0u);
                        mbar_arrive(bar(isv ? C::B_VFACT + (jt & 1) : C::B_KFACT + (jt & 3)));
                    }
                }
                // NaN rows of a V tile that some row does not see are zeroed and noted
                const uint32_t bad4 = ((nan >> 7) * 0x01020408u) >> 24 & 15u;
                if (isv && fix) {
                    // lane l holds rows 4l..: word q of the tile is lanes 8q .. 8q + 7
                    uint32_t word = bad4 << (4 * (lane & 7));
                    word |= __shfl_xor_sync(0xffffffffu, word, 1);
                    word |= __shfl_xor_sync(0xffffffffu, word, 2);
                    word |= __shfl_xor_sync(0xffffffffu, word, 4);
                    if (w == 0 && (lane & 7) == 0) s_poison[(nfix % kPoison) * 4 + (lane >> 3)] = word;
                }
                const uint32_t zero4 = isv ? (~in4 & 15u) | (fix ? bad4 : 0u) : 0u;
                const bool zeros = __any_sync(0xffffffffu, zero4 != 0u);
                // (opaque to the compiler, which would make two loops: 150 -> 158 us for 8 x
                // 32 drafts over 24K)
                int scaled = wide ? 0 : -1;
                asm("" : "+r"(scaled));
                constexpr int BATCH = T == 256 ? 2 : 4;  // groups whose loads are in flight
#pragma unroll 1
                for (int g0 = 0; g0 < ROWS / 8; g0 += BATCH) {
                    uint4 code[BATCH][C::HALVES];
                    uint32_t by[BATCH];
#pragma unroll
                    for (int gi = 0; gi < BATCH; ++gi) {
                        by[gi] = sc[w * ROWS + (g0 + gi) * 8 + rq];
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h)
                            code[gi][h] = *reinterpret_cast<const uint4 *>(
                                src + (g0 + gi) * 8 * C::ROWB + so[h]);
                    }
#pragma unroll
                    for (int gi = 0; gi < BATCH; ++gi) {
                        // 2^(byte - top) in f16 (at least 2^-15 for what is attended), or
                        // 1 where each key has its own scale; a NaN for a NaN row
                        const int d = ((int)by[gi] - (int)top) & scaled;
                        uint32_t f = d >= -14 ? (uint32_t)(15 + min(d, 0)) << 10
                                     : d == -15 ? 1u << 9
                                                : 0u;
                        if (by[gi] == kScaleNaN) f = 0x7fffu;
                        f |= f << 16;
                        bool zero = false;
                        if (zeros) {
                            const int r = w * ROWS + (g0 + gi) * 8 + rq;
                            zero = (__shfl_sync(0xffffffffu, zero4, r >> 2) >> (r & 3)) & 1u;
                        }
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h) {
                            const uint4 cw = code[gi][h];
                            uint32_t y[8];
                            e4m3_to_f16(cw.x, y[0], y[1]);
                            e4m3_to_f16(cw.y, y[2], y[3]);
                            e4m3_to_f16(cw.z, y[4], y[5]);
                            e4m3_to_f16(cw.w, y[6], y[7]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = f16x2_mul(y[e], f);
                            if (zero)
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = 0u;
                            uint8_t *o = dst + h * C::HALF + (g0 + gi) * 1024;
                            *reinterpret_cast<uint4 *>(o + do0) = make_uint4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<uint4 *>(o + do1) = make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (isv && fix) mbar_arrive(bar(C::B_POISON + nfix % kPoison));
                    mbar_arrive(bar((isv ? C::B_VFULL : C::B_KFULL) + s));
                    mbar_arrive(bar(C::B_REMPTY + rs));
                }
            }
            if (fix) ++nfix;
        }
        release(ns);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == C::W_MMA) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, C::TMEM);
    }
}

// ---------------------------------------------------------------------------
// merge of the partitions, sink, cast: one warp per (draft, query head)
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 128;

__global__ void __launch_bounds__(kMergeThreads)
tree_merge_kernel(const TreeParams p, int rows) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.z, t = blockIdx.y;
    const int h = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const Req rq = request(p, b, false);
    if (t >= rq.q_len || h >= p.num_qo_heads) return;
    // the row group's place on the line, and the CTA groups it meets: the first
    // left the second slot of its two, the others their first
    const int D = p.head_dim, G = p.group, g = h / G;
    const int row = t * G + (h - g * G), rg = row / rows;
    const int tiles = cost_of(p, rq, rows).tiles;
    const long long s = p.line[b] + (long long)rg * tiles, share = p.line[p.batch];
    const int first = (int)(s / share), last = (int)((s + tiles - 1) / share);
    if (first == last) return;  // one CTA had all of it
    const int n = last - first + 1;
    const int r = row - rg * rows;
    auto slot = [&](int i) {
        return (int64_t)(i == 0 ? 2 * first + 1 : 2 * (first + i)) * p.num_kv_heads + g;
    };
    auto lse_of = [&](int i) { return p.part_lse[slot(i) * rows + r]; };
    const float sink = p.sink ? p.sink[h] * kLog2e : kNegInf;
    float M = sink;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, lse_of(i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float Ms = M == kNegInf ? 0.f : M;
    float sum = 0.f;
    for (int i = lane; i < n; i += 32) sum += exp2f(lse_of(i) - Ms);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float lam = sum + exp2f(sink - Ms);
    const float inv = lam == 0.f ? 0.f : 1.f / lam;
    const int64_t unit = (int64_t)(rq.q_start + t) * p.num_qo_heads + h;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + unit * D;
    for (int c = 4 * lane; c < D; c += 128) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float w = exp2f(lse_of(i) - Ms) * inv;
            const float4 v = reinterpret_cast<const float4 *>(
                p.part_o)[(slot(i) * (D / 4) + c / 4) * rows + r];
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
        *reinterpret_cast<uint2 *>(out + c) =
            make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    }
    if (p.lse_out && lane == 0) p.lse_out[unit] = lam == 0.f ? kNegInf : (Ms + log2f(lam)) * kLn2;
}

template <int T, bool KV8, int X>
cudaError_t launch_one(const TreeParams &p, const CUtensorMap *tk, const CUtensorMap *tv,
                       cudaStream_t stream) {
    using C = Cfg<T, KV8, X>;
    auto kern = tree_kernel<T, KV8, X>;
    cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void *>(kern), C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.num_kv_heads * p.groups), dim3(C::THREADS), (size_t)C::SMEM,
                      stream, p, *tk, *tv);
}

template <bool KV8>
cudaError_t launch_kv(const TreeParams &p, const CUtensorMap *tk, const CUtensorMap *tv,
                      cudaStream_t stream) {
    if (p.head_dim > 128) return launch_one<256, KV8, 1>(p, tk, tv, stream);
    if (p.row_tiles > 1)
        return p.head_dim <= 64 ? launch_one<64, KV8, 2>(p, tk, tv, stream)
                                : launch_one<128, KV8, 2>(p, tk, tv, stream);
    return p.head_dim <= 64 ? launch_one<64, KV8, 1>(p, tk, tv, stream)
                            : launch_one<128, KV8, 1>(p, tk, tv, stream);
}

}  // namespace

cudaError_t launch_tree(const TreeParams &p, const CUtensorMap *tmap_k,
                        const CUtensorMap *tmap_v, cudaStream_t stream) {
    cudaError_t e = p.k_scale ? launch_kv<true>(p, tmap_k, tmap_v, stream)
                              : launch_kv<false>(p, tmap_k, tmap_v, stream);
    if (e != cudaSuccess) return e;
    constexpr int kHeads = kMergeThreads / 32;
    return launch_pdl(tree_merge_kernel,
                      dim3((p.num_qo_heads + kHeads - 1) / kHeads, p.max_seqlen_q, p.batch),
                      dim3(kMergeThreads), 0, stream, p,
                      p.head_dim <= 128 && p.row_tiles > 1 ? 2 * kTile : kTile);
}

}  // namespace pkv
