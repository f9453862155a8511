// The matrix products of the dense feed-forward operators on gfx950 MFMA
// (v_mfma_f32_32x32x16 of bf16 or fp16), fp32 accumulators.
//
//   acc[m][n] = sum_k A(m, k) B(n, k), each operand k- or m/n-contiguous
//
// A block of WM x WN waves owns BM x BN outputs and walks K in tiles of BK.
//   DMA      16-byte aligned rows: global memory -> LDS directly
//            (buffer_load ... lds), no operand passes through a register; a ring
//            of NS stages keeps NS - 1 k-tiles in flight ahead of the MFMAs
//   register any alignment and any width: 16-byte loads at element alignment
//            into registers, NSTAGE sets of them in flight ahead; LDS stores
//            between the MFMAs of the k-tile before
// Past the last row the last row is read again (its results are not stored);
// past the last k both operands are zeros.
//
// LDS holds a k-contiguous operand as rows of BK / 8 16-byte chunks, XOR-swizzled
// (rswz: 16 rows of one chunk touch 16 distinct bank groups), read as one
// fragment of 8 k per ds_read_b128.  An m-contiguous operand keeps its global layout, k rows of BM elements, and is transposed on
// the way to registers by ds_read_b64_tr_b16 (16 lanes fetch 4 k x 16 m and each
// gets the 4 k of its m); the 64-byte groups of a row are XORed with k & 3, so
// that the four k rows of such a fetch lie in distinct banks.  So the backward
// products read dz, W and x as they are, without a transposing pass.
//
// fp32 operands are split on their way to LDS into three bf16 parts, x = h + m + l
// exactly (h: the upper 8 bits of the significand; m: the rest rounded to 8; l: what
// is left), and six products make one: hh' + hm' + mh' + hl' + lh' + mm'.  What is
// left out, ml' + lm' + ll', is below 2^-22 |x x'| and of either sign, as the
// rounding of an fp32 sum of a few terms is.  Six bf16 MFMAs of 16 k take 192 cycles
// of the matrix pipe, the eight fp32 ones they replace 512.  An infinity or NaN goes
// into l alone, which meets only h', and so gives what it should; an infinity's h is
// 2^-100 of its sign, for the other operand's infinity in l' to meet (beside a finite x'
// it adds 2^-100 x' to an infinity).  Parts below bf16's subnormals are lost, 2^-134 |x'|
// per product.
//
// Output goes out by rows through LDS, 8 columns per lane: bias, activation,
// residual and the gated product are applied there to the fp32 sums, and loads
// and stores are 16 bytes wide.
//
// Bound by the matrix pipe and the loads beside it: 8192 x 16384 of K 4096 in bf16,
// 903 to 941 us (1217 to 1168 TFLOP/s; with every operand tile in L2 833 us, without any
// loads 725); gated 4096 x 2 x 1024 of K 4096 62 to 65 us (1112 to 1062 TFLOP/s).  fp32
// by splitting the operands, LDS and MFMAs together: 1000 x 1024 of K 2048 38 to 40 us
// (107 TFLOP/s), 2293 x 2814 of K 3776 forward and backward 159 (the library's fp32
// products reach 152).
#pragma once

#include <type_traits>

#include "dense_device.h"

namespace ecf {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

template <class E>
__device__ __forceinline__ f32x16_t mfma16(u32x4_t a, u32x4_t b, f32x16_t c);
template <>
__device__ __forceinline__ f32x16_t mfma16<BF16>(u32x4_t a, u32x4_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16_t mfma16<F16>(u32x4_t a, u32x4_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

template <>
__device__ __forceinline__ f32x16_t mfma16<F32>(u32x4_t a, u32x4_t b, f32x16_t c)  // of parts
{
    return mfma16<BF16>(a, b, c);
}

// The blocks of one product, in one dimension: splits of K x output tiles.  Block b
// runs on XCD b % 8, each with its own L2: an XCD gets a contiguous run of tiles,
// eight tile rows high and as many columns as it takes, so blocks running together
// share operand tiles in that L2 (4, 16 and 32 rows: within 1%, or slower).
struct DenseGrid {
    int tiles_m, tiles_n;  // tiles_m: of both halves
    int half_tiles;        // tiles_m of one half
    int splits;
    float *partial;  // splits > 1: fp32 sums [split][half or projection][M][np]
    int64_t np;
    __host__ __device__ int blocks() const { return tiles_m * tiles_n * splits; }
    __device__ __forceinline__ void locate(int b, int &split, int &half, int &mt, int &nt) const
    {
        const int total = blocks(), x = b & 7, q = total >> 3, r = total & 7;
        int i = x * q + min(x, r) + (b >> 3);
        split = i / (tiles_m * tiles_n);
        i -= split * tiles_m * tiles_n;
        const int panel = i / (8 * tiles_n), h = min(8, tiles_m - panel * 8);
        i -= panel * 8 * tiles_n;
        nt = i / h;
        mt = panel * 8 + i - nt * h;
        half = mt >= half_tiles ? 1 : 0;
        mt -= half * half_tiles;
    }
    __device__ __forceinline__ int64_t partial_at(const DenseGemm &g, int split, int plane, int64_t m) const
    {
        return (((int64_t)split * (g.gated ? 2 : g.mhalves) + plane) * g.M + m) * np;
    }
};

// ---- epilogue on 8 columns of one row -------------------------------------------------

// Bias of columns n..n+7, of each projection.
template <class E, bool GATED>
__device__ __forceinline__ void load_bias(const DenseGemm &g, int n, float bias[GATED ? 2 : 1][8])
{
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q)
        if (g.bias[q] && n < g.N)
            load8<E>(g.bias[q], n, g.N - n, bias[q]);
}

// Residual of columns n..n+7 of row m.
template <class E>
__device__ __forceinline__ void load_res(const DenseGemm &g, int64_t m, int n, float res[8])
{
    if (m >= g.M || n >= g.N)
        return;
    if (g.out_dtype == ECF_F32)
        load8<F32>(row_at<F32>(g.res, m * g.ldres), n, g.N - n, res);
    else
        load8<E>(row_at<E>(g.res, m * g.ldres), n, g.N - n, res);
}

// Saved sums, activation ACT, gated product or residual, and the output of columns
// n..n+7 of row m; z[q] are the fp32 sums (q = 1: the up projection).  PLAIN: the
// sums are the output, as in the backward products, whose code stays small for it.
// They are multiplied by `mul` first (backward products in fp16).
template <class E, bool GATED, bool PLAIN, int ACT>
__device__ __forceinline__ void epilogue8(const DenseGemm &g, int half, int64_t m, int n, float z[GATED ? 2 : 1][8],
                                          const float bias[GATED ? 2 : 1][8], const float res[8], float mul = 1.f)
{
    const int cnt = g.N - n;
    if (cnt <= 0 || m >= g.M)
        return;
    void *out = g.out[half];
    float y[8];
    if constexpr (PLAIN) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = std::is_same<E, F16>::value ? z[0][j] * mul : z[0][j];
    } else {
#pragma unroll
        for (int q = 0; q < (GATED ? 2 : 1); ++q) {
            if (g.bias[q]) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    z[q][j] += bias[q][j];
            }
            if (g.save[q])
                store8<E>(row_at<E>(g.save[q], m * g.ldsave), n, cnt, z[q], g.stream_out);
        }
        if (!out)
            return;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[j] = act_value(z[0][j], ACT);
            if constexpr (GATED)
                y[j] *= z[1][j];
        }
        if (!GATED && g.res) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] += res[j];
        }
    }
    if (g.out_dtype == ECF_F32)
        store8<F32>(row_at<F32>(out, m * g.ldout), n, cnt, y, g.stream_out);
    else
        store8<E>(row_at<E>(out, m * g.ldout), n, cnt, y, g.stream_out);
}

// What undoes the scale of row m of A (DenseGemm::unscale), in products that may have one.
template <class E, bool BT>
__device__ __forceinline__ float unscale_of(const DenseGemm &g, int half, int64_t m)
{
    if constexpr (std::is_same<E, F16>::value && BT)
        return g.unscale ? g.unscale[(int64_t)half * g.M + min(m, (int64_t)g.M - 1)] : 1.f;
    return 1.f;
}

// ---- operand tiles ----------------------------------------------------------------------

namespace gemm {

constexpr uint32_t kNowhere = 0x80000000u;  // a buffer offset past every resource: reads zeros, touches no memory

typedef uint32_t lds_addr;
__device__ __forceinline__ lds_addr lds_of(const void *p)
{
    return (lds_addr)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// 16 bytes per lane from global memory straight into LDS, lane l's at lds + 16 l.
// Written as assembly: through the builtin the compiler makes the next LDS read
// wait for the load, although that read is of the other stage.  The load has no
// register result; the k-tile's end waits for it (stage_ready).
__device__ __forceinline__ void dma16(u32x4_t rsrc, uint32_t voff, lds_addr lds)
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff),
                 "s"(rsrc)
                 : "memory");
#endif
}

__device__ __forceinline__ u32x4_t rsrc_of(const void *base)
{
    const uint64_t b = (uint64_t)(uintptr_t)base;
    // base, no stride, 2 GiB - 1 of range, raw 32-bit data format
    u32x4_t r = {(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, 0x7fffffffu, 0x00020000u};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[i]);
    return r;
}

// At most N of this wave's loads are still under way (the k-tiles behind the next
// one) and its LDS accesses are done: meet the other waves.
template <int N>
__device__ __forceinline__ void stage_ready()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// k-contiguous tiles: the XOR of the chunks of row r.  16 rows of one chunk then
// lie in 16 distinct 16-byte bank groups of 256 bytes (rows of 128 bytes: two
// rows per 256, eight chunks each; rows of 64 bytes: four rows, four chunks).
template <int BK>
__device__ __forceinline__ int rswz(int r)
{
    return BK == 64 ? (r & 7) ^ ((r >> 3) & 1) : (r >> 2) & 3;
}
// m-contiguous tiles: the XOR of the 16-byte chunks of k row k (64-byte groups
// over 4 k rows; rows of 128 bytes put two k rows side by side, so there it takes
// k / 2).
template <int ROWS>
__device__ __forceinline__ int kswz(int k)
{
    return ROWS >= 128 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
}

// 8 fp32 values to three chunks of bf16 parts.  `odd` becomes infinite or NaN if one
// of the values is (or is near 2^90); their k-tile is stored again through split8_odd.
__device__ __forceinline__ void split8(const u32x4_t v[2], u32x4_t part[3], float &odd)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t u0 = v[j >> 1][2 * (j & 1)], u1 = v[j >> 1][2 * (j & 1) + 1];
        const float x0 = __uint_as_float(u0), x1 = __uint_as_float(u1);
        part[0][j] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);  // the upper halves
        const float r0 = x0 - __uint_as_float(u0 & 0xffff0000u), r1 = x1 - __uint_as_float(u1 & 0xffff0000u);
        const bf16x2_t m = {(__bf16)r0, (__bf16)r1};
        const uint32_t mw = __builtin_bit_cast(uint32_t, m);
        part[1][j] = mw;
        // at most 8 bits are left: their upper half is all of them
        const float l0 = r0 - bf_lo(mw), l1 = r1 - bf_hi(mw);
        part[2][j] = __builtin_amdgcn_perm(__float_as_uint(l1), __float_as_uint(l0), 0x07060302u);
        odd = __builtin_fmaf(l0, l1, odd);  // what is left of an infinity or NaN is NaN
    }
}

__device__ __forceinline__ void split8_odd(const u32x4_t v[2], u32x4_t part[3])
{
    float odd = 0.f;
    split8(v, part, odd);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t u = v[j >> 2][j & 3];
        if ((u & 0x7f800000u) == 0x7f800000u) {
            const uint32_t keep = j & 1 ? 0x0000ffffu : 0xffff0000u;
            const uint32_t top = (u & 0x7fffffu) ? u | 0x400000u : u;  // a NaN stays one in 16 bits
            // h of an infinity: +-2^-100 in bf16
            const uint32_t h = (u & 0x7fffffu) ? 0u : (u >> 16 & 0x8000u) | 0x0d80u;
            part[0][j >> 1] = (part[0][j >> 1] & keep) | (j & 1 ? h << 16 : h);
            part[1][j >> 1] &= keep;
            part[2][j >> 1] = (part[2][j >> 1] & keep) | (j & 1 ? top & 0xffff0000u : top >> 16);
        }
    }
}

// One operand's tile of ROWS rows (m or n) x BK k.  T: m-contiguous in memory.
// ES: bytes per element in memory; fp32 tiles (register path) lie in LDS as three
// planes of bf16 parts.
template <bool T, bool DMA, int ROWS, int NTH, int BK, int ES, int SETS>
struct Tile {
    static_assert(ES == 2 || !DMA, "fp32 is split on its way to LDS");
    static constexpr int W = ES / 2;  // 16-byte registers per chunk of 8 elements
    static constexpr int CPR = T ? ROWS / 8 : BK / 8;  // chunks per LDS row
    static constexpr int NL = ROWS * BK / 8 / NTH;     // 16-byte loads per thread and k-tile
    static constexpr int STEP = NTH / CPR;             // LDS rows between a thread's loads
    static constexpr int RPW = 64 / CPR;               // LDS rows that one load of a wave covers (not T)
    static_assert(ROWS * BK / 8 % NTH == 0 && NL >= 1, "tile too small for the block");
    static_assert(STEP % (T ? 4 : 16) == 0, "a thread's rows share the swizzle");

    uint32_t off[NL];  // byte offsets of this thread's chunks from the k-tile's base
    int row, chunk;    // the first of this thread's LDS rows, and its chunk in all of them
    int valid;         // T: elements of the chunk that exist (up to 8, none if <= 0)
    // register path: the chunks of SETS k-tiles and the k each had left.  No load sits
    // behind a branch (at the branch's end the compiler would wait for it): a lane
    // with nothing to load reads the tile's first 8 elements.  What lies
    // past the last m is of no account (no output that is stored sees it), what lies
    // past the last k has to be zero.  So a chunk cut by the last m reads on into the
    // next row; in the operand's last row it is the 8 elements that end at the edge,
    // which store_again() moves down, as for a chunk cut by the last k.  The launcher
    // sends operands with rows of under 8 elements elsewhere.
    const char *first;  // the operand's first element, for k-tiles past the end
    int rows;           // rows from the tile's first on
    int kl[SETS];
    u32x4_t reg[SETS][DMA ? 1 : NL][W];

    // `rows` rows from the tile's first on, row stride ld (elements); rowmap turns a
    // tile row into a row relative to the base (clamped to the last one)
    template <class F>
    __device__ __forceinline__ void init(int tid, int rows_, const void *first_, int64_t ld, F rowmap)
    {
        row = tid / CPR;
        first = (const char *)first_;
        rows = rows_;
        if constexpr (!T) {
            chunk = (tid % CPR) ^ rswz<BK>(row);
            valid = 8;
#pragma unroll
            for (int q = 0; q < NL; ++q)
                off[q] = (uint32_t)(rowmap(row + STEP * q) * ld * ES) + chunk * (8 * ES);
        } else {
            chunk = (tid % CPR) ^ kswz<ROWS>(row);
            valid = rows - chunk * 8;
#pragma unroll
            for (int q = 0; q < NL; ++q)
                off[q] = (uint32_t)((row + STEP * q) * ld * ES) + chunk * (8 * ES);
        }
    }

    // Start loading the k-tile at `base` with kleft k still to come (over BK, or
    // none and less: zeros).  PAIR: tile rows r with bit 5 set come from base2 (the
    // up projection); the rows that one load of a wave covers agree on that bit.
    static constexpr bool second(int q, int wave) { return (STEP * q + RPW * wave) >> 5 & 1; }

    // DMA: load q of the k-tile
    template <bool PAIR>
    __device__ __forceinline__ void issue(u32x4_t rs, u32x4_t rs2, int q, int kleft, lds_addr lds, int wave)
    {
        static_assert(!PAIR || (!T && RPW <= 32 && 32 % RPW == 0), "a wave's rows agree on bit 5");
        const bool in = T ? valid > 0 && row + STEP * q < kleft : chunk * 8 < kleft;
        dma16(PAIR && second(q, wave) ? rs2 : rs, in ? off[q] : kNowhere, lds + (q * NTH + 64 * wave) * 16);
    }

    // register path: a whole k-tile into set S
    template <bool PAIR, int S>
    __device__ __forceinline__ void load(const void *base, const void *base2, int kleft, int wave)
    {
        // Offsets from 8 elements before the tile, so that none is negative and each
        // load is a scalar base and one 32-bit register.  back(n): a chunk of n
        // elements is taken from 8 - n elements further down.
        auto back = [](int n) { return (uint32_t)min(max(8 - n, 0), 8) * ES; };
        const bool last = !T || kleft <= BK;  // else cut chunks read on into the next row
        const int n = T ? valid : kleft - chunk * 8;
        const uint32_t shift = 8 * ES - (last ? back(n) : 0u);
        const uint32_t none = kleft <= 0 ? 8u * ES : 8 * ES - (last ? back(T ? rows : kleft) : 0u);
        const char *b1 = (kleft > 0 ? (const char *)base : first) - 8 * ES;
        const char *b2 = (kleft > 0 ? (const char *)base2 : first) - 8 * ES;
        kl[S] = kleft;
#pragma unroll
        for (int q = 0; q < NL; ++q) {
            const bool in = n > 0 && (!T || row + STEP * q < kleft);
            const char *p = (PAIR && second(q, wave) ? b2 : b1) + (in ? off[q] + shift : none);
            if constexpr (ES == 2) {
                reg[S][q][0] = ((const any128x2 *)p)->v;
            } else {
                reg[S][q][0] = __builtin_bit_cast(u32x4_t, ((const any128x4 *)p)->v);
                reg[S][q][1] = __builtin_bit_cast(u32x4_t, ((const any128x4 *)(p + 16))->v);
            }
        }
    }

    // does the k-tile in set S reach over the last k, or hold cut chunks of the last row?
    template <int S>
    __device__ __forceinline__ bool edge() const
    {
        return kl[S] < BK || (T && rows < ROWS && kl[S] == BK);
    }

    // register path: chunk q of set S to its stage, as if nothing were cut or odd (see split8)
    template <int S>
    __device__ __forceinline__ void store(int q, char *stage, int tid, float &odd) const
    {
        u32x4_t *at = (u32x4_t *)stage + q * NTH + tid;
        if constexpr (ES == 2) {
            *at = reg[S][q][0];
        } else {
            u32x4_t part[3];
            split8(reg[S][q], part, odd);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                at[p * (ROWS * BK / 8)] = part[p];
        }
    }

    // The whole k-tile again: cut chunks moved down, zeros past the edge, and
    // infinities and NaNs where they belong.  Apart from store(), so that store() is
    // straight code between MFMAs.
    template <int S>
    __device__ __forceinline__ void store_again(char *stage, int tid) const
    {
#pragma unroll
        for (int q = 0; q < NL; ++q) {
            u32x4_t v[W];
#pragma unroll
            for (int w = 0; w < W; ++w)
                v[w] = reg[S][q][w];
            // as load() took it: only in the last row's k-tile are chunks cut by the last m moved
            const int n = !T ? kl[S] - chunk * 8 : row + STEP * q >= kl[S] ? 0 : kl[S] <= BK ? valid : 8;
            const int s = min(8, max(0, 8 - n));
            if (s & 7) {
                if constexpr (ES == 2) {
                    v[0] = shift_down16(v[0], s & 7);
                } else {
#pragma unroll
                    for (int b = 4; b >= 1; b >>= 1)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (s & b)
                                v[j >> 2][j & 3] = j + b < 8 ? v[(j + b) >> 2][(j + b) & 3] : 0u;
                }
            }
#pragma unroll
            for (int w = 0; w < W; ++w)
                v[w] = s >= 8 ? u32x4_t{0, 0, 0, 0} : v[w];
            u32x4_t *at = (u32x4_t *)stage + q * NTH + tid;
            if constexpr (ES == 2) {
                *at = v[0];
            } else {
                u32x4_t part[3];
                split8_odd(v, part);
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    at[p * (ROWS * BK / 8)] = part[p];
            }
        }
    }
};

// Where a lane finds its fragments of an operand in a stage.  Fragment f: rows
// r0 + 32 f + (lane & 31); step ks: k chunk BK / 16 (lane >> 5) + ks, 8 k.
template <bool T, int ROWS, int F, int BK>
struct Frag {
    static constexpr int NK = BK / 16;
    uint32_t at[T ? F : NK];
    __device__ __forceinline__ void init(int lane, int r0, int ks0)  // read()'s step 0 is ks0
    {
        const int g = lane >> 5;
        if constexpr (!T) {
            const int r = r0 + (lane & 31);
#pragma unroll
            for (int ks = 0; ks < NK; ++ks)
                at[ks] = r * (BK * 2) + ((NK * g + ((ks0 + ks) & (NK - 1))) ^ rswz<BK>(r)) * 16;
        } else {
            const int i = lane & 15, k = BK / 2 * g + (i >> 2);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int m = r0 + 32 * f + (lane & 16) + (i & 3) * 4;
                at[f] = (k + 8 * ks0) * (ROWS * 2) + (((m >> 3) ^ kswz<ROWS>(k)) * 16) + (m & 4) * 2;
            }
        }
    }
    __device__ __forceinline__ u32x4_t read(const char *stage, int f, int ks) const
    {
        if constexpr (!T) {
            return *(const u32x4_t *)(stage + at[ks] + f * 32 * (BK * 2));
        } else {
            u32x4_t v = {0, 0, 0, 0};
#if defined(__HIP_DEVICE_COMPILE__)
            typedef __attribute__((address_space(3))) s16x4_t lds4;
            const char *p = stage + at[f] + ks * 8 * (ROWS * 2);
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + 4 * (ROWS * 2)));
            const uint64_t a = __builtin_bit_cast(uint64_t, lo), b = __builtin_bit_cast(uint64_t, hi);
            v = u32x4_t{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
#endif
            return v;
        }
    }
};

}  // namespace gemm

// LDS of a block: the stages, which the output staging takes over at the end.
template <class E, bool DMA, int BM, int BN, int WM, int WN, int BK, int NSTAGE>
constexpr int gemm_lds_bytes()
{
    constexpr int in = (DMA ? NSTAGE : 2) * (BM + BN) * BK * 2 * (sizeof(typename E::raw) == 4 ? 3 : 1);
    constexpr int out = WM * WN * 32 * (64 + 4) * 4;
    return in > out ? in : out;
}

// Block `block` of a product: one (split, output tile), see DenseGrid.  KW: groups of
// WM x WN waves that share each k-tile's steps; their sums are joined at the end.  Two
// groups for the fp32 64 x 64 tile, whose LDS leaves room for one block: with two waves
// per SIMD one splits operands while the other multiplies (K 4096: 1.22 -> 1.00 us per
// k-tile of 64).
template <class E, bool AT, bool BT, bool GATED, bool DMA, int BM, int BN, int WM, int WN, int BK, int NSTAGE, int KW>
__device__ __forceinline__ void gemm_block(const DenseGemm &g, const DenseGrid &gr, int block, char *lds)
{
    using namespace gemm;
    constexpr int NW = WM * WN, NTH = 64 * NW * KW, RM = BM / WM, RN = BN / WN, FM = RM / 32, FN = RN / 32;
    static_assert(BK % (32 * KW) == 0, "two sets of fragments take turns");
    static_assert(KW <= 2 && (KW == 1 || (FM == 1 && FN == 1)), "a group's sums fit the stages' LDS");
    static_assert(DMA || NSTAGE <= 2, "one or two register sets");
    static_assert(FM >= 1 && (FN == 1 || FN % 2 == 0) && (!GATED || (!BT && WN * FN % 2 == 0)), "wave tile");
    constexpr int NS = DMA ? NSTAGE : 2, SETS = DMA ? 1 : NSTAGE;
    constexpr int ES = sizeof(typename E::raw), NP = ES == 4 ? 3 : 1;      // planes of parts
    constexpr int PA = BM * BK * 2, PB = BN * BK * 2, SA = PA * NP, SB = PB * NP;  // bytes per plane and stage
    constexpr bool MATES = GATED && FN == 1;  // a wave has the gate or the up columns only, its neighbour the others
    constexpr int PITCH = (FN >= 2 || GATED ? 64 : 32) + 4;  // fp32 per row of the output staging

    int split, half, mt, nt;
    gr.locate(block, split, half, mt, nt);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = KW > 1 ? wave / NW : 0, gwave = KW > 1 ? wave % NW : wave, wm = gwave / WN, wn = gwave % WN;
    const int m0 = mt * BM, n0 = nt * (GATED ? BN / 2 : BN);
    const int mrows = min(BM, g.M - m0);

    Tile<AT, DMA, BM, NTH, BK, ES, SETS> ta;
    Tile<BT, DMA, BN, NTH, BK, ES, SETS> tb;
    const int nrows = GATED ? 0 : g.N - n0, nlast = g.N - 1 - n0;
    ta.init(tid, g.M - m0, g.a[0], g.lda, [&](int r) { return (int64_t)min(r, mrows - 1); });
    // gated: 64 tile rows are 32 of the gate projection, then the same 32 of the up projection
    tb.init(tid, nrows, g.b[0], g.ldb,
            [&](int r) { return (int64_t)min(GATED ? (r >> 6) * 32 + (r & 31) : r, nlast); });
    Frag<AT, BM, FM, BK> fa;
    Frag<BT, BN, FN, BK> fb;
    constexpr int NK = BK / 16 / KW;  // a group's steps of each k-tile
    fa.init(lane, wm * RM, group * NK);
    fb.init(lane, wn * RN, group * NK);

    f32x16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.f;

    const int kper = (g.K + BK - 1) / BK;  // k-tiles per segment
    const int64_t kall = (int64_t)kper * g.ksegs;
    const int kb = (int)(kall * split / gr.splits), ke = (int)(kall * (split + 1) / gr.splits);
    // Operand addresses of the block's first k, and the bytes from one k-tile to the
    // next.  Held in scalar registers: left alone, the compiler reads the pointers
    // from the kernel's arguments again in every k-tile and waits for them.
    const char *pa[2], *pb[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        pa[q] = (const char *)g.a[AT ? half : q] + (AT ? (int64_t)m0 : (int64_t)m0 * g.lda) * ES;
        pb[q] = (const char *)g.b[q] + (BT ? (int64_t)n0 : (int64_t)n0 * g.ldb) * ES;
        asm volatile("" : "+s"(pa[q]), "+s"(pb[q]));
    }
    const int64_t stepa = (AT ? g.lda : 1) * (ES * BK), stepb = (BT ? g.ldb : 1) * (ES * BK);
    constexpr int NLA = decltype(ta)::NL, NLD = NLA + decltype(tb)::NL;
    // k-tile kt: past the end nothing is loaded (zeros)
    struct Src {
        const char *a, *b, *b2;
        int kleft;
    };
    auto source = [&](int kt) __attribute__((always_inline)) {
        const bool seg = kt >= kper;
        const int k = seg ? kt - kper : kt;
        return Src{(seg && !AT ? pa[1] : pa[0]) + k * stepa, (seg && !GATED ? pb[1] : pb[0]) + k * stepb,
                   pb[1] + k * stepb, kt < ke ? g.K - k * BK : 0};
    };
    // DMA: load q of the NLD loads of a k-tile towards `stage`
    auto issue = [&](const Src &s, int stage, int q) __attribute__((always_inline)) {
        const lds_addr to = lds_of(lds) + stage * (SA + SB);
        if (q < NLA)
            ta.template issue<false>(rsrc_of(s.a), rsrc_of(s.a), q, s.kleft, to, wave);
        else
            tb.template issue<GATED>(rsrc_of(s.b), rsrc_of(GATED ? s.b2 : s.b), q - NLA, s.kleft, to + SA, wave);
    };
    // register path: k-tile kt into set S, and piece q of set S to `stage`
    auto load_reg = [&](int kt, auto set) __attribute__((always_inline)) {
        constexpr int S = decltype(set)::value;
        const Src s = source(kt);
        ta.template load<false, S>(s.a, s.a, s.kleft, wave);
        tb.template load<GATED, S>(s.b, s.b2, s.kleft, wave);
        // issue the loads here, ahead of the MFMAs they travel under
        asm volatile("" ::: "memory");
    };
    float odd = 0.f;
    auto put = [&](int q, int stage, auto set) __attribute__((always_inline)) {
        constexpr int S = decltype(set)::value;
        if (q < NLA)
            ta.template store<S>(q, lds + stage * (SA + SB), tid, odd);
        else
            tb.template store<S>(q - NLA, lds + stage * (SA + SB) + SA, tid, odd);
    };
    auto put_again = [&](int stage, auto set) __attribute__((always_inline)) {
        constexpr int S = decltype(set)::value;
        if (ta.template edge<S>() || tb.template edge<S>() || (NP == 3 && !(fabsf(odd) < __builtin_huge_valf()))) {
            ta.template store_again<S>(lds + stage * (SA + SB), tid);
            tb.template store_again<S>(lds + stage * (SA + SB) + SA, tid);
            odd = 0.f;
        }
    };
    // Two sets of fragments: step ks + 1 (or the next k-tile's step 0) is read under
    // the MFMAs of step ks.
    u32x4_t av[2][FM][NP], bv[2][FN][NP];
    auto fetch = [&](int stage, int ks, int set, int f) __attribute__((always_inline)) {
        const char *sa = lds + stage * (SA + SB), *sb = sa + SA;
#pragma unroll
        for (int p = 0; p < NP; ++p)
            if (f < FN)
                bv[set][f][p] = fb.read(sb + p * PB, f, ks);
            else
                av[set][f - FN][p] = fa.read(sa + p * PA, f - FN, ks);
    };
    auto fetch_all = [&](int stage) __attribute__((always_inline)) {
#pragma unroll
        for (int f = 0; f < FM + FN; ++f)
            fetch(stage, 0, 0, f);
    };
    // The MFMAs of the fragments in `set`.  Before MFMA i: fragments of step ks of
    // `stage` into the other set, spread over the MFMAs so that they have the rest of
    // the step to arrive, and extra(i) (global loads, or LDS stores).  The scheduling barriers keep
    // this order: left alone, the compiler moves the reads behind the last MFMAs.
    constexpr int MF = FM * FN;
    auto step = [&](int set, int stage, int ks, auto extra) __attribute__((always_inline)) {
        auto reads = [&](int i) __attribute__((always_inline)) {
#pragma unroll
            for (int f = i * (FM + FN) / MF; f < (i + 1) * (FM + FN) / MF; ++f)
                fetch(stage, ks, set ^ 1, f);
            extra(i);
        };
        if constexpr (NP == 1) {
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                reads(i);
                acc[i / FN][i % FN] = mfma16<E>(av[set][i / FN][0], bv[set][i % FN][0], acc[i / FN][i % FN]);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            // six products, the small ones first; neighbours write different sums, so
            // that none waits for the one before it
            constexpr int PA_[6] = {1, 0, 2, 0, 1, 0}, PB_[6] = {1, 2, 0, 1, 0, 0};
#pragma unroll
            for (int x = 0; x < 6 * MF; ++x) {
                if (x % 6 == 0)
                    reads(x / 6);
                const int i = x % MF, p = x / MF;
                acc[i / FN][i % FN] = mfma16<E>(av[set][i / FN][PA_[p]], bv[set][i % FN][PB_[p]], acc[i / FN][i % FN]);
                if (x % 6 == 5)
                    __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    if (kb < ke) {
        // The k-tile's last step: its fragments are in registers, so this stage is
        // done with; once the next k-tile has landed for every wave, its first
        // fragments are read under the last step's MFMAs.
        if constexpr (DMA) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const Src s = source(kb + i);
#pragma unroll
                for (int q = 0; q < NLD; ++q)
                    issue(s, i, q);
            }
            stage_ready<(NS - 1) * NLD>();
            fetch_all(0);
            int stage = 0;
            for (int kt = kb; kt < ke; ++kt) {
                const Src s = source(kt + NS);
#pragma unroll
                for (int ks = 0; ks < NK - 1; ++ks)
                    step(ks & 1, stage, ks + 1, [](int) {});
                const int next = stage + 1 == NS ? 0 : stage + 1;
                stage_ready<(NS - 2) * NLD>();
                step((NK - 1) & 1, next, 0, [&](int i) __attribute__((always_inline)) {
#pragma unroll
                    for (int q = i * NLD / MF; q < (i + 1) * NLD / MF; ++q)
                        issue(s, stage, q);
                });
                stage = next;
            }
            stage_ready<0>();
        } else {
            // k-tile kb + i goes through register set i % SETS into stage i % 2: loaded
            // while k-tile i - 1 - SETS is multiplied, stored while i - 1 is
            load_reg(kb, std::integral_constant<int, 0>{});
#pragma unroll
            for (int q = 0; q < NLD; ++q)
                put(q, 0, std::integral_constant<int, 0>{});
            put_again(0, std::integral_constant<int, 0>{});
            load_reg(kb + 1, std::integral_constant<int, 1 % SETS>{});
            if constexpr (SETS == 2)
                load_reg(kb + 2, std::integral_constant<int, 0>{});
            stage_ready<63>();
            fetch_all(0);
            int stage = 0;
            // k-tile kt; the next one waits in register set S
            auto tile = [&](int kt, auto set) __attribute__((always_inline)) {
                constexpr int PIECES = MF * (NK - 1);
#pragma unroll
                for (int ks = 0; ks < NK - 1; ++ks)
                    step(ks & 1, stage, ks + 1, [&](int i) __attribute__((always_inline)) {
                        const int at = ks * MF + i;
#pragma unroll
                        for (int q = at * NLD / PIECES; q < (at + 1) * NLD / PIECES; ++q)
                            put(q, stage ^ 1, set);
                    });
                put_again(stage ^ 1, set);
                load_reg(kt + 1 + SETS, set);
                stage_ready<63>();
                stage ^= 1;
                step((NK - 1) & 1, stage, 0, [](int) {});
            };
            for (int kt = kb; kt < ke; kt += SETS) {
                tile(kt, std::integral_constant<int, 1 % SETS>{});
                if constexpr (SETS == 2)
                    if (kt + 1 < ke)
                        tile(kt + 1, std::integral_constant<int, 0>{});
            }
            stage_ready<63>();
        }
    }

    if constexpr (KW > 1) {
        // the second group's sums to the first, which stores the output
        f32x4_t *sums = (f32x4_t *)lds + gwave * 256 + lane;
        if (group) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sums[64 * e] = f32x4_t{acc[0][0][4 * e], acc[0][0][4 * e + 1], acc[0][0][4 * e + 2], acc[0][0][4 * e + 3]};
        }
        __syncthreads();
        if (!group) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[0][0][e] += sums[64 * (e >> 2)][e & 3];
        }
        __syncthreads();
    }

    // Output through LDS: each wave puts 32 rows x (up to) 64 columns of fp32 sums
    // in its own buffer and takes them back by rows.  A wave's LDS accesses
    // complete in order, so only the compiler has to be kept from reordering them.
    // The loop over the groups stays a loop: unrolled, the epilogue's code is fetched
    // from memory by every block (8192 x 16384 bf16 outputs of K 128 took 350 us, as
    // a loop 133).  Bias and residual of a group are loaded ahead of its LDS round trip.
    constexpr int CB = FN >= 2 ? 2 : 1, GROUPS = FM * (FN / CB);
    constexpr int LPR = (GATED ? 32 : 32 * CB) / 8;  // lanes per output row
    // (two waves that hold the two projections of the same columns share a buffer,
    // and take half its rows each)
    float *eb = (float *)lds + (MATES ? gwave / 2 : gwave) * 32 * PITCH;
    const int ecol = MATES ? (wn & 1) * 32 : 0, erow = MATES ? (wn & 1) * 16 : 0;
    const bool partial = gr.splits > 1;
    constexpr int PASSES = MATES ? 1 : 32 * LPR / 64, Q = GATED ? 2 : 1;
    if (KW > 1 && group) {
        for (int i = 0; MATES && i < 2 * GROUPS; ++i)
            __syncthreads();  // the ones below
        return;
    }
#pragma unroll 1
    for (int grp = 0; grp < GROUPS; ++grp) {
        const int r0 = wm * RM + grp / (FN / CB) * 32 + erow + lane / LPR, c = (lane % LPR) * 8;
        const int c0 = MATES ? wn / 2 * 32 : GATED ? (wn * RN + grp % (FN / CB) * 64) / 2 : wn * RN + grp % (FN / CB) * 64;
        const int n = n0 + c0 + c;
        constexpr bool PLAIN = BT;
        float bias[Q][8], res[GATED || PLAIN ? 1 : PASSES][8], mul[PASSES];
        if (PLAIN && !partial) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p)
                mul[p] = unscale_of<E, PLAIN>(g, half, m0 + r0 + p * (64 / LPR));
        }
        if (!PLAIN && !partial) {
            load_bias<E, GATED>(g, n, bias);
            if (!GATED && g.res) {
#pragma unroll
                for (int p = 0; p < PASSES; ++p)
                    load_res<E>(g, m0 + r0 + p * (64 / LPR), n, res[GATED || PLAIN ? 0 : p]);
            }
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
            if (grp == i) {
#pragma unroll
                for (int j = 0; j < CB; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        eb[((e >> 2) * 8 + (lane >> 5) * 4 + (e & 3)) * PITCH + ecol + j * 32 + (lane & 31)] =
                            acc[i / (FN / CB)][i % (FN / CB) * CB + j][e];
            }
        asm volatile("" ::: "memory");
        if constexpr (MATES)
            __syncthreads();
        auto take = [&](int p, float z[Q][8]) __attribute__((always_inline)) {
            const float *at = eb + (erow + p * (64 / LPR) + lane / LPR) * PITCH + c;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const f32x4_t lo = *(const f32x4_t *)(at + q * 32), hi = *(const f32x4_t *)(at + q * 32 + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[q][e] = lo[e], z[q][4 + e] = hi[e];
            }
        };
        if (partial) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int64_t m = m0 + r0 + p * (64 / LPR);
                float z[Q][8];
                take(p, z);
                if (m < g.M && n < g.N) {
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        store8<F32>(gr.partial, gr.partial_at(g, split, GATED ? q : half, m) + n, 8, z[q]);
                }
            }
        } else if constexpr (PLAIN) {
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                float z[Q][8];
                take(p, z);
                epilogue8<E, GATED, true, ECF_ACT_NONE>(g, half, m0 + r0 + p * (64 / LPR), n, z, bias, res[0], mul[p]);
            }
        } else {
            with_act(g.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    float z[Q][8];
                    take(p, z);
                    epilogue8<E, GATED, false, decltype(act)::value>(g, half, m0 + r0 + p * (64 / LPR), n, z, bias,
                                                                     res[GATED || PLAIN ? 0 : p]);
                }
            });
        }
        if constexpr (MATES)
            __syncthreads();
    }
}

// Waves per SIMD asked of the register allocator: two, but one where a wave's own
// tile of sums takes more than half the registers.
#define ECF_GEMM_BOUNDS __launch_bounds__(64 * WM * WN * KW, BM / WM * (BN / WN) > 128 * 64 ? 1 : 2)

template <class E, bool AT, bool BT, bool GATED, bool DMA, int BM, int BN, int WM, int WN, int BK, int NSTAGE, int KW>
__global__ ECF_GEMM_BOUNDS void k_gemm(DenseGemm g, DenseGrid gr)
{
    __shared__ __attribute__((aligned(16))) char lds[gemm_lds_bytes<E, DMA, BM, BN, WM, WN, BK, NSTAGE>()];
    gemm_block<E, AT, BT, GATED, DMA, BM, BN, WM, WN, BK, NSTAGE, KW>(g, gr, (int)blockIdx.x, lds);
}

// Column sums over the row blocks, in order, and zeros where there is no row block
// at all: block b takes 64 columns, its first four waves a quarter of the row blocks
// each.  red: 1 KiB of LDS.
__device__ __forceinline__ void colsum_block(const DenseColsum &s, int b, float *red)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t c = (int64_t)b * 64 + lane, cols = (int64_t)s.n * s.I;
    float v = 0.f;
    if (c < cols && w < 4)
#pragma unroll 8
        for (int64_t r = w; r < s.row_blocks; r += 4)
            v += s.partial[r * cols + c];
    if (w < 4)
        red[w * 64 + lane] = v;
    __syncthreads();
    if (w || c >= cols)
        return;
    void *out = c < s.I ? s.out[0] : s.out[1];
    if (out)
        store_el(out, c < s.I ? c : c - s.I, (red[lane] + red[64 + lane]) + (red[128 + lane] + red[192 + lane]),
                 s.out_dtype);
}

// The two products of a backward pass, dz W and dz^T x, in one launch: each alone
// often leaves CUs idle, and neither needs the other.  The blocks of the longer
// reduction come first, the column sums' last (as a launch of their own: 3.5 us more).
template <class E, bool DMA, int BM, int BN, int WM, int WN, int BK, int NSTAGE, int KW>
__global__ ECF_GEMM_BOUNDS void k_gemm_pair(DenseGemm gx, DenseGrid grx, DenseGemm gw, DenseGrid grw, DenseColsum sums,
                                              int x_first)
{
    __shared__ __attribute__((aligned(16))) char lds[gemm_lds_bytes<E, DMA, BM, BN, WM, WN, BK, NSTAGE>()];
    const int nx = grx.blocks(), nw = grw.blocks(), b = (int)blockIdx.x;
    if (b >= nx + nw)
        colsum_block(sums, b - nx - nw, (float *)lds);
    else if (x_first ? b < nx : b >= nw)
        gemm_block<E, false, true, false, DMA, BM, BN, WM, WN, BK, NSTAGE, KW>(gx, grx, x_first ? b : b - nw, lds);
    else
        gemm_block<E, true, true, false, DMA, BM, BN, WM, WN, BK, NSTAGE, KW>(gw, grw, x_first ? b - nx : b, lds);
}

// Joins the splits of a product, in order, and applies its epilogue: one thread
// per 8 columns of a row.
template <class E, bool GATED>
__global__ __launch_bounds__(256) void k_dense_join(DenseGemm g, DenseGrid gr)
{
    const int64_t per = gr.np / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per * g.M * g.mhalves)
        return;
    const int64_t row = i / per;
    const int n = (int)(i - row * per) * 8, half = row >= g.M ? 1 : 0;
    const int64_t m = row - (half ? g.M : 0);
    float z[GATED ? 2 : 1][8] = {}, bias[GATED ? 2 : 1][8], res[8];
    load_bias<E, GATED>(g, n, bias);
    if (!GATED && g.res)
        load_res<E>(g, m, n, res);
#pragma unroll 4
    for (int s = 0; s < gr.splits; ++s)
#pragma unroll
        for (int q = 0; q < (GATED ? 2 : 1); ++q) {
            float v[8];
            load8<F32>(gr.partial, gr.partial_at(g, s, GATED ? q : half, m) + n, 8, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                z[q][j] += v[j];
        }
    if constexpr (std::is_same<E, F16>::value && !GATED) {
        const float mul = unscale_of<E, true>(g, half, m);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            z[0][j] *= mul;
    }
    with_act(g.act, [&](auto act) __attribute__((always_inline)) {
        epilogue8<E, GATED, false, decltype(act)::value>(g, half, m, n, z, bias, res);
    });
}

}  // namespace ecf
