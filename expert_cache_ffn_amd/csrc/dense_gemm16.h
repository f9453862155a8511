// The 16-bit (bf16, fp16) matrix products of the dense feed-forward operators on
// gfx950 MFMA (v_mfma_f32_32x32x16), fp32 accumulators.
//
//   acc[m][n] = sum_k A(m, k) B(n, k), each operand k- or m/n-contiguous
//
// A block of WM x WN waves owns BM x BN outputs and walks K in tiles of 64, two
// LDS stages: while the MFMAs of one k-tile run, the next one's operands travel.
//   DMA      16-byte aligned rows: global memory -> LDS directly
//            (buffer_load ... lds), no operand passes through a register
//   register any alignment and any width: 16-byte loads at element alignment
//            into registers at the top of a k-tile, LDS stores at its end
// Past the last row the last row is read again (its results are not stored);
// past the last k both operands are zeros.
//
// LDS holds a k-contiguous operand as rows of eight 16-byte chunks, chunk c of
// row r at c ^ (r & 7) ^ bit 3 of r (16 rows of one chunk touch 16 distinct
// bank groups), read as one fragment of 8 k per ds_read_b128.  An m-contiguous
// operand keeps its global layout, k rows of BM elements, and is transposed on
// the way to registers by ds_read_b64_tr_b16 (16 lanes fetch 4 k x 16 m and each
// gets the 4 k of its m); the 64-byte groups of a row are XORed with k & 3, so
// that the four k rows of such a fetch lie in distinct banks.  So the backward
// products read dz, W and x as they are, without a transposing pass.
//
// Output goes out by rows through LDS, 8 columns per lane: bias, activation,
// residual and the gated product are applied there to the fp32 sums, and loads
// and stores are 16 bytes wide where alignment allows.
#pragma once

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

// The blocks of one product, in one dimension: splits of K x output tiles.  Block b
// runs on XCD b % 8, each with its own L2: an XCD gets a contiguous run of tiles,
// eight tile rows high and as many columns as it takes, so blocks running together share operand
// tiles in that L2.
struct DenseGrid {
    int tiles_m, tiles_n;  // tiles_m: of both halves
    int half_tiles;        // tiles_m of one half
    int ktiles, splits;
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

// p[0..8) of a row: 16-byte accesses where the launcher found every row aligned
// (vec), else one element at a time, n of them.
template <class E>
__device__ __forceinline__ void load8(const void *p, int64_t i, int n, bool vec, float v[8])
{
    const typename E::raw *q = (const typename E::raw *)p + i;
    if (vec && n >= 8) {
        if constexpr (sizeof(typename E::raw) == 4) {
            const f32x4_t a = *(const f32x4_t *)q, b = *(const f32x4_t *)(q + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = a[j], v[4 + j] = b[j];
        } else {
            const u32x4_t a = *(const u32x4_t *)q;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = E::to_f((uint16_t)(a[j] & 0xffffu));
                v[2 * j + 1] = E::to_f((uint16_t)(a[j] >> 16));
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = j < n ? E::to_f(q[j]) : 0.f;
}

template <class E>
__device__ __forceinline__ void store8(void *p, int64_t i, int n, bool vec, const float v[8])
{
    typename E::raw *q = (typename E::raw *)p + i;
    if (vec && n >= 8) {
        if constexpr (sizeof(typename E::raw) == 4) {
            *(f32x4_t *)q = f32x4_t{v[0], v[1], v[2], v[3]};
            *(f32x4_t *)(q + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
        } else {
            u32x4_t a;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                a[j] = (uint32_t)E::from_f(v[2 * j]) | (uint32_t)E::from_f(v[2 * j + 1]) << 16;
            *(u32x4_t *)q = a;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n)
            q[j] = E::from_f(v[j]);
}

// Bias, saved sums, activation, gated product or residual, and the output of
// columns n..n+7 of row m; z[q] are the fp32 sums (q = 1: the up projection).
template <class E, bool GATED>
__device__ __forceinline__ void epilogue8(const DenseGemm &g, int half, int64_t m, int n, float z[GATED ? 2 : 1][8])
{
    const int cnt = g.N - n;
    if (cnt <= 0)
        return;
#pragma unroll
    for (int q = 0; q < (GATED ? 2 : 1); ++q) {
        if (g.bias[q]) {
            float bv[8];
            load8<E>(g.bias[q], n, cnt, g.vec_bias, bv);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                z[q][j] += bv[j];
        }
        if (g.save[q])
            store8<E>(g.save[q], m * g.ldsave + n, cnt, g.vec_save, z[q]);
    }
    void *out = g.out[half];
    if (!out)
        return;
    float y[8];
    // the activation is uniform: one switch for the eight values
    if (g.act == ECF_ACT_NONE) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = z[0][j];
    } else if (g.act == ECF_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = act_value(z[0][j], ECF_ACT_SILU);
    } else if (g.act == ECF_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = act_value(z[0][j], ECF_ACT_GELU);
    } else if (g.act == ECF_ACT_GELU_TANH) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = act_value(z[0][j], ECF_ACT_GELU_TANH);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = act_value(z[0][j], ECF_ACT_RELU);
    }
    if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] *= z[1][j];
    } else if (g.res) {
        float r[8];
        if (g.out_dtype == ECF_F32)
            load8<F32>(g.res, m * g.ldres + n, cnt, g.vec_res, r);
        else
            load8<E>(g.res, m * g.ldres + n, cnt, g.vec_res, r);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] += r[j];
    }
    if (g.out_dtype == ECF_F32)
        store8<F32>(out, m * g.ldout + n, cnt, g.vec_out, y);
    else
        store8<E>(out, m * g.ldout + n, cnt, g.vec_out, y);
}

// ---- operand tiles ----------------------------------------------------------------------

namespace g16 {

constexpr int BK = 64;
constexpr uint32_t kNowhere = 0x80000000u;  // a buffer offset past every resource: reads zeros, touches no memory

typedef uint32_t lds_addr;
__device__ __forceinline__ lds_addr lds_of(const void *p)
{
    return (lds_addr)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// 16 bytes per lane from global memory straight into LDS, lane l's at lds + 16 l.
// Written as assembly: through the builtin the compiler makes the next LDS read
// wait for the load, although that read is of the other stage.  The load has no
// register result; the k-tile's end waits for it (stage_end).
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

// the next stage has landed and this stage is read: wait for this wave's loads and LDS reads, meet the others
__device__ __forceinline__ void stage_end()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// m-contiguous tiles: the XOR of the 16-byte chunks of k row k (64-byte groups over 4 k rows; rows of 128 bytes
// put two k rows side by side, so there it takes k / 2)
template <int ROWS>
__device__ __forceinline__ int kswz(int k)
{
    return ROWS >= 128 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
}

struct __attribute__((packed, aligned(2))) u128_any {
    u32x4_t v;
};

// One operand's tile of ROWS rows (m or n) x 64 k.  T: m-contiguous in memory.
template <bool T, bool DMA, int ROWS, int NTH>
struct Tile {
    static constexpr int NL = ROWS * 8 / NTH;  // 16-byte loads per thread and k-tile
    static constexpr int CPR = T ? ROWS / 8 : 8;  // chunks per LDS row
    static constexpr int KSTEP = NTH * 8 / ROWS;  // T: k rows between a thread's loads
    static_assert(ROWS * 8 % NTH == 0 && NL >= 1, "tile too small for the block");
    static_assert(!T || KSTEP % 4 == 0, "a thread's k rows share the swizzle");

    uint32_t off[NL];  // byte offsets of this thread's chunks from the k-tile's base
    int row, chunk;    // T: first k row and chunk; else: chunk of every row
    int valid;         // T: elements of the chunk that exist (0..8); else unused
    u32x4_t reg[DMA ? 1 : NL];

    // `rows` real rows from the tile's first on, row stride ld (elements); rowmap
    // turns a tile row into a row relative to the base (before clamping)
    template <class F>
    __device__ __forceinline__ void init(int tid, int rows, int64_t ld, F rowmap)
    {
        if constexpr (!T) {
            row = tid >> 3;
            chunk = (tid & 7) ^ (row & 7) ^ ((row >> 3) & 1);
            valid = 8;
#pragma unroll
            for (int q = 0; q < NL; ++q) {
                const int64_t r = rowmap(row + (NTH / 8) * q);
                off[q] = (uint32_t)(r * ld * 2) + chunk * 16;
            }
        } else {
            row = tid / CPR;
            chunk = (tid % CPR) ^ kswz<ROWS>(row);
            valid = max(0, min(8, rows - chunk * 8));
#pragma unroll
            for (int q = 0; q < NL; ++q)
                off[q] = (uint32_t)((row + KSTEP * q) * ld * 2) + chunk * 16;
        }
    }

    // Start loading the k-tile at `base` with kleft k still to come (may be over 64).
    // PAIR: tile rows r with bit 5 set come from base2 (the up projection); the 8
    // rows that one load of a wave covers agree on that bit.
    template <bool PAIR = false>
    __device__ __forceinline__ void load(const void *base, int kleft, lds_addr lds, int wave,
                                         const void *base2 = nullptr)
    {
        auto second = [&](int q) { return PAIR && ((((NTH / 8) * q + 8 * wave) >> 5) & 1); };
        if constexpr (DMA) {
            const u32x4_t rs = rsrc_of(base), rs2 = PAIR ? rsrc_of(base2) : rs;
            if constexpr (!T) {
                const bool in = chunk * 8 < kleft;
#pragma unroll
                for (int q = 0; q < NL; ++q)
                    dma16(second(q) ? rs2 : rs, in ? off[q] : kNowhere, lds + (q * NTH + 64 * wave) * 16);
            } else {
#pragma unroll
                for (int q = 0; q < NL; ++q)
                    dma16(rs, valid && row + KSTEP * q < kleft ? off[q] : kNowhere, lds + (q * NTH + 64 * wave) * 16);
            }
        } else {
            const int n = T ? valid : kleft - chunk * 8;
            if (T ? n >= 8 && kleft >= BK : n >= 8) {
#pragma unroll
                for (int q = 0; q < NL; ++q)
                    reg[q] = ((const u128_any *)((const char *)(second(q) ? base2 : base) + off[q]))->v;
            } else {
#pragma unroll
                for (int q = 0; q < NL; ++q) {
                    const bool in = !T || row + KSTEP * q < kleft;
                    const uint16_t *p = (const uint16_t *)((const char *)(second(q) ? base2 : base) + off[q]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t lo = 0, hi = 0;
                        if (in && 2 * j < n)
                            lo = p[2 * j];
                        if (in && 2 * j + 1 < n)
                            hi = p[2 * j + 1];
                        reg[q][j] = lo | hi << 16;
                    }
                }
            }
        }
    }

    // register path: the loaded k-tile to its stage
    __device__ __forceinline__ void store(u32x4_t *stage, int tid)
    {
        if constexpr (!DMA) {
#pragma unroll
            for (int q = 0; q < NL; ++q)
                stage[q * NTH + tid] = reg[q];
        }
    }
};

// Where a lane finds its fragments of an operand in a stage.  Fragment f: rows
// r0 + 32 f + (lane & 31); step ks: k chunk 4 (lane >> 5) + ks, 8 k.
template <bool T, int ROWS, int F>
struct Frag {
    uint32_t at[T ? F : 4];
    __device__ __forceinline__ void init(int lane, int r0)
    {
        const int g = lane >> 5;
        if constexpr (!T) {
            const int r = r0 + (lane & 31);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                at[ks] = (r * 8 + ((4 * g + ks) ^ (r & 7) ^ ((r >> 3) & 1))) * 16;
        } else {
            const int i = lane & 15, k = 32 * g + (i >> 2);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int m = r0 + 32 * f + (lane & 16) + (i & 3) * 4;
                at[f] = k * (ROWS * 2) + (((m >> 3) ^ kswz<ROWS>(k)) * 16) + (m & 4) * 2;
            }
        }
    }
    __device__ __forceinline__ u32x4_t read(const char *stage, int f, int ks) const
    {
        if constexpr (!T) {
            return *(const u32x4_t *)(stage + at[ks] + f * 32 * 128);
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

}  // namespace g16

// grid: 1-D, one block per (split, output tile); see DenseGrid.
template <class E, bool AT, bool BT, bool GATED, bool DMA, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_gemm16(DenseGemm g,
                                                                                                   DenseGrid gr)
{
    using namespace g16;
    constexpr int NW = WM * WN, NTH = 64 * NW, RM = BM / WM, RN = BN / WN, FM = RM / 32, FN = RN / 32;
    static_assert(FM >= 1 && FN >= 1 && (!GATED || (FN == 2 && !BT)), "wave tile");
    constexpr int SA = BM * 128, SB = BN * 128;  // bytes per stage
    constexpr int PITCH = (FN >= 2 ? 64 : 32) + 4;  // fp32 per row of the output staging
    static_assert(NW * 32 * PITCH * 4 <= 2 * (SA + SB), "output staging");
    __shared__ __attribute__((aligned(16))) char lds[2 * (SA + SB)];

    int split, half, mt, nt;
    gr.locate(blockIdx.x, split, half, mt, nt);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int m0 = mt * BM, n0 = nt * (GATED ? BN / 2 : BN);
    const int mrows = min(BM, g.M - m0);

    Tile<AT, DMA, BM, NTH> ta;
    Tile<BT, DMA, BN, NTH> tb;
    ta.init(tid, g.M - m0, g.lda, [&](int r) { return (int64_t)min(r, mrows - 1); });
    if constexpr (GATED) {
        // 64 tile rows: 32 of the gate projection, then the same 32 of the up projection
        tb.init(tid, 0, g.ldb, [&](int r) { return (int64_t)min((r >> 6) * 32 + (r & 31), g.N - 1 - n0); });
    } else {
        tb.init(tid, g.N - n0, g.ldb, [&](int r) { return (int64_t)min(r, g.N - 1 - n0); });
    }
    Frag<AT, BM, FM> fa;
    Frag<BT, BN, FN> fb;
    fa.init(lane, wm * RM);
    fb.init(lane, wn * RN);

    f32x16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.f;

    const int kper = (g.K + BK - 1) / BK;  // k-tiles per segment
    const int kb = (int)((int64_t)gr.ktiles * split / gr.splits), ke = (int)((int64_t)gr.ktiles * (split + 1) / gr.splits);
    auto load = [&](int kt, int stage) __attribute__((always_inline)) {
        const int seg = kt >= kper ? 1 : 0, k0 = (kt - seg * kper) * BK;
        const char *a = (const char *)(AT ? (half ? g.a[1] : g.a[0]) : (seg ? g.a[1] : g.a[0]));
        const char *b = (const char *)(seg ? g.b[1] : g.b[0]);
        a += (AT ? (int64_t)k0 * g.lda + m0 : (int64_t)m0 * g.lda + k0) * 2;
        const int64_t bo = (BT ? (int64_t)k0 * g.ldb + n0 : (int64_t)n0 * g.ldb + k0) * 2;
        ta.load(a, g.K - k0, lds_of(lds) + stage * SA, wave);
        if constexpr (GATED)
            tb.template load<true>(b + bo, g.K - k0, lds_of(lds) + 2 * SA + stage * SB, wave, (const char *)g.b[1] + bo);
        else
            tb.load(b + bo, g.K - k0, lds_of(lds) + 2 * SA + stage * SB, wave);
        // issue the loads here, ahead of the MFMAs they travel under
        asm volatile("" ::: "memory");
    };
    auto put = [&](int stage) __attribute__((always_inline)) {
        ta.store((u32x4_t *)(lds + stage * SA), tid);
        tb.store((u32x4_t *)(lds + 2 * SA + stage * SB), tid);
    };
    auto body = [&](int stage) __attribute__((always_inline)) {
        const char *sa = lds + stage * SA, *sb = lds + 2 * SA + stage * SB;
        // fragments of step ks + 1 are read under the MFMAs of step ks; the
        // scheduling barriers keep the compiler from reading all four steps ahead,
        // which takes more registers than there are
        u32x4_t av[2][FM], bv[2][FN];
        auto fetch = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
                bv[ks & 1][j] = fb.read(sb, j, ks);
#pragma unroll
            for (int i = 0; i < FM; ++i)
                av[ks & 1][i] = fa.read(sa, i, ks);
        };
        fetch(0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            if (ks < 3)
                fetch(ks + 1);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = mfma16<E>(av[ks & 1][i], bv[ks & 1][j], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (kb < ke) {
        load(kb, 0);
        put(0);
        stage_end();
        int stage = 0;
        for (int kt = kb; kt + 1 < ke; ++kt) {
            load(kt + 1, stage ^ 1);
            body(stage);
            stage ^= 1;
            put(stage);
            stage_end();
        }
        body(stage);
    }
    __syncthreads();

    // Output through LDS: each wave puts 32 rows x (up to) 64 columns of fp32 sums
    // in its own buffer and takes them back by rows.  A wave's LDS accesses
    // complete in order, so only the compiler has to be kept from reordering them.
    float *eb = (float *)lds + wave * 32 * PITCH;
    const bool partial = gr.splits > 1;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int jp = 0; jp < FN; jp += 2) {
            constexpr int CB = FN >= 2 ? 2 : 1;
            asm volatile("" ::: "memory");
#pragma unroll
            for (int j = 0; j < CB; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    eb[((e >> 2) * 8 + (lane >> 5) * 4 + (e & 3)) * PITCH + j * 32 + (lane & 31)] = acc[i][jp + j][e];
            asm volatile("" ::: "memory");
            constexpr int LPR = (GATED ? 32 : 32 * CB) / 8;  // lanes per output row
#pragma unroll
            for (int p = 0; p < 32 * LPR / 64; ++p) {
                const int r = p * (64 / LPR) + lane / LPR, c = (lane % LPR) * 8;
                const int64_t m = m0 + wm * RM + i * 32 + r;
                const int n = n0 + (GATED ? wn * 32 : wn * RN + jp * 32) + c;
                float z[GATED ? 2 : 1][8];
#pragma unroll
                for (int q = 0; q < (GATED ? 2 : 1); ++q) {
                    const f32x4_t lo = *(const f32x4_t *)(eb + r * PITCH + q * 32 + c);
                    const f32x4_t hi = *(const f32x4_t *)(eb + r * PITCH + q * 32 + c + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[q][e] = lo[e], z[q][4 + e] = hi[e];
                }
                if (m >= g.M)
                    continue;
                if (!partial) {
                    epilogue8<E, GATED>(g, half, m, n, z);
                } else if (n < g.N) {
#pragma unroll
                    for (int q = 0; q < (GATED ? 2 : 1); ++q)
                        store8<F32>(gr.partial, gr.partial_at(g, split, GATED ? q : half, m) + n, 8, true, z[q]);
                }
            }
            asm volatile("" ::: "memory");
        }
    }
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
    float z[GATED ? 2 : 1][8] = {};
    for (int s = 0; s < gr.splits; ++s)
#pragma unroll
        for (int q = 0; q < (GATED ? 2 : 1); ++q) {
            float v[8];
            load8<F32>(gr.partial, gr.partial_at(g, s, GATED ? q : half, m) + n, 8, true, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                z[q][j] += v[j];
        }
    epilogue8<E, GATED>(g, half, m, n, z);
}

// How a product is cut: the tile, the splits of K, and whether operands can go
// straight to LDS.
struct DensePlan {
    int tile;  // index into the launcher's tiles
    int splits;
    bool dma;
};

}  // namespace ecf
