// fi_lattn.hip -- linear attention with a decay per head (fi_lattn_*).
//
// Per row b, key/value head n and position t, lam = exp(ld[n]):
//     S[t] = lam S[t-1] + k[t] v[t]^T,   o[t][h] = scale S[t]^T q[t][h].
#include <algorithm>
#include <type_traits>

#include "fi_opdev.hpp"

namespace fi {

// ------------------------------------------------------------ recurrent form
// One position: a workgroup has dk x 32 of one (row, head)'s state, thread (r,
// c) = (tid / 8, tid % 8) the columns 4c .. 4c+3 of the slice and the rows r,
// r + 32, ...: columns of S never meet, so slices need no exchange, and rows
// of the slice are whole lines of memory.
// Bound by the state, read and written once: 200 rows x 8 heads of 128 x 128
// (214 MB with q, k, v and o, 32 query heads) take 41 to 47 us, 4.6 to 5.3 TB/s,
// what a large copy reaches (4.9); 71 us before the state's loads were 16 bytes
// each and all asked for before the position's own arrive.  One row: 3.8 us, a
// launch and two trips to memory.
constexpr int kRecThreads = 256;
constexpr int kRecCols = 32;
constexpr int kRecRows = kRecThreads / (kRecCols / 4);   // rows in one sweep
constexpr int kRecHeads = 4;                             // query heads at a time

template <bool BF16, int RPT, bool VEC>
__global__ __launch_bounds__(kRecThreads) void k_lattn_step(LattnCall a) {
    constexpr int ROWS = kRecRows * RPT, WAVES = kRecThreads / kWave;
    __shared__ float ks[ROWS], qs[kRecHeads][ROWS];
    __shared__ __align__(16) float vs[kRecCols], red[WAVES][kRecHeads][kRecCols];   // read in 16-byte units
    const int tid = threadIdx.x, c = tid % (kRecCols / 4), r = tid / (kRecCols / 4);
    const int slices = (a.dv + kRecCols - 1) / kRecCols;
    const int64_t b = blockIdx.x / slices / a.Hkv;
    const int n = blockIdx.x / slices % a.Hkv, col0 = blockIdx.x % slices * kRecCols;
    const int dk = a.dk, dv = a.dv, G = a.G;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool in = slot >= 0 && slot < a.n_slots;
    const bool here = in && (!a.lens || a.lens[b] > 0);   // (a prompt's row may be empty)
    const int col = col0 + 4 * c, left = dv - col;   // columns of the state from the thread's first on

    // everything that the position reads is asked for at once
    float* const sp = in ? a.state + (slot * a.Hkv + n) * dk * (int64_t)dv + r * dv + col : nullptr;
    V4 S[RPT] = {};
    if (in && !a.fresh) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (r + i * kRecRows < dk) {
                const FI_GLOBAL float* p = gmem(sp + i * kRecRows * dv);
                if constexpr (VEC) {
                    if (left > 0) S[i] = *reinterpret_cast<const FI_GLOBAL V4*>(p);
                } else
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left) S[i][j] = p[j];
            }
    }
    const int64_t kb = b * a.k.row + n * a.k.head, vb = b * a.v.row + n * a.v.head, qb = b * a.q.row + (int64_t)n * G * a.q.head;
    const auto load_q = [&](int g0) {
        const int gn = G - g0 < kRecHeads ? G - g0 : kRecHeads;
        for (int i = tid; i < gn * ROWS; i += kRecThreads)
            qs[i / ROWS][i % ROWS] = here && i % ROWS < dk ? get_io<BF16>(a.q.p, qb + (g0 + i / ROWS) * a.q.head + i % ROWS) : 0.f;
    };
    for (int i = tid; i < ROWS; i += kRecThreads) ks[i] = here && i < dk ? get_io<BF16>(a.k.p, kb + i) : 0.f;
    if (tid < kRecCols) vs[tid] = here && col0 + tid < dv ? get_io<BF16>(a.v.p, vb + col0 + tid) : 0.f;
    load_q(0);
    const float em1 = here ? expm1f(a.ld[n]) : 0.f;   // lam - 1
    const bool kept = here || (in && a.fresh);        // the state changes
    __syncthreads();

    // S + (lam - 1) S rather than lam S: the rounding of lam (up to 2^-25 of S
    // a step, always to one side) would add up over long memories
    const V4 v = *smem_ptr(reinterpret_cast<const V4*>(&vs[4 * c]));
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const float k = ks[r + i * kRecRows];
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] = fmaf(k, v[j], fmaf(em1, S[i][j], S[i][j]));
        if (kept && r + i * kRecRows < dk) {
            FI_GLOBAL float* p = gmem(sp + i * kRecRows * dv);
            if constexpr (VEC) {
                if (left > 0) *reinterpret_cast<FI_GLOBAL V4*>(p) = S[i];
            } else
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) p[j] = S[i][j];
        }
    }
    for (int g0 = 0; g0 < G; g0 += kRecHeads) {
        const int gn = G - g0 < kRecHeads ? G - g0 : kRecHeads;
        if (g0) {
            __syncthreads();
            load_q(g0);
            __syncthreads();
        }
#pragma unroll
        for (int g = 0; g < kRecHeads; ++g) {
            if (g >= gn) break;
            V4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float q = qs[g][r + i * kRecRows];
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = fmaf(q, S[i][j], p[j]);
            }
#pragma unroll
            for (int d = 8; d < kWave; d <<= 1)
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] += __shfl_xor(p[j], d);
            if (tid % kWave < 8) *smem_ptr(reinterpret_cast<V4*>(&red[tid / kWave][g][4 * c])) = p;
        }
        __syncthreads();
        for (int i = tid; i < gn * kRecCols; i += kRecThreads) {
            const int g = i / kRecCols, j = i % kRecCols;
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) o += red[w][g][j];
            if (col0 + j < dv) put_io<BF16>(a.o.p, b * a.o.row + (n * G + g0 + g) * a.o.head + col0 + j, here ? a.scale * o : 0.f);
        }
    }
}

hipError_t launch_lattn_step(const LattnCall& c, hipStream_t st) {
    const bool small = c.dk <= 4 * kRecRows, vec = c.dv % 4 == 0;   // the state's rows are whole 16-byte units
    const dim3 grid((unsigned)((c.dv + kRecCols - 1) / kRecCols * c.Hkv * c.B));   // B Hkv <= kLattnMaxRows
    const auto go = [&](auto bf, auto rpt) {
        constexpr bool BF16 = decltype(bf)::value;
        constexpr int RPT = decltype(rpt)::value;
        if (vec) k_lattn_step<BF16, RPT, true><<<grid, kRecThreads, 0, st>>>(c);
        else k_lattn_step<BF16, RPT, false><<<grid, kRecThreads, 0, st>>>(c);
    };
    using std::integral_constant;
    if (c.io_bf16 && small) go(std::true_type{}, integral_constant<int, 4>{});
    else if (c.io_bf16) go(std::true_type{}, integral_constant<int, 8>{});
    else if (small) go(std::false_type{}, integral_constant<int, 4>{});
    else go(std::false_type{}, integral_constant<int, 8>{});
    return hipGetLastError();
}

// ------------------------------------------------------------ chunked form
// A workgroup takes a segment of positions of one (row, head) and a slice of
// DVS columns of S, chunk by chunk; each of its waves has 16 of the columns.
// With Q, K, V a chunk's rows, E the state before it and i, j < C:
//     O = scale (diag(lam^{i+1}) Q E + P V),  P[i][j] = lam^{i-j} q_i . k_j, j <= i
//     S = lam^C E + K^T diag(lam^{C-1-j}) V
// A row's first chunk is filled from the back (zero rows in front), so that
// every later one is whole and ends on the row's last position.
//
// Long rows of few heads are split into segments: OUT = false forms every
// segment's state from zero, k_lattn_scan joins them into the states before the
// segments, OUT = true starts from those.  That reads K and V twice; carrying
// the state from segment to segment instead would leave a row to its slices.
//
// Split: a wave's columns of S stay in its registers from chunk to chunk, and
// S is the operand of both of its products as it lies there; the waves meet
// only in P, whose tiles they share out.  Waves with 32 columns (operands used
// twice, half the waves) took 303 us where these took 297, and 132 where these
// took 91 (ragged rows, four heads a group; both with one part of P and E).
//
// Roundings (bf16): the operands of the products are bf16, so P and, in Q E, E
// enter as two bf16 parts each, off by 2^-16 of them at most: o is the formula's value
// rounded once (0.0001 of its norm from that; with one part each 0.0025, which is more
// than the rounding itself, and what the step does to the same state would be another
// number; 64K x 16 heads 397 -> 429 us, ragged rows 122 -> 130, one row of 77 8.3 -> 8.7).
// V's decayed rows go into S in three parts, exactly, so that S keeps fp32's
// precision over any number of chunks.
//
// Measured: 16 heads of 128 x 128, 65536 positions, bf16: 429 us (1.07 GB once:
// 2.5 TB/s): local states 115 to 135, scan 15, outputs 293 to 350.  The outputs keep
// the vector units busy 51%, LDS 35% and the matrix cores 32% of the time with 3.1
// waves a SIMD: none of them is full, and a wave goes through a chunk one phase after
// the other (operands to LDS, P, O, S, four barriers), which two workgroups on a CU
// overlap in part.  fp32, two rows of 4001, 16 heads of 64 x 64: 61 us, outputs 41
// (matrix cores 41%).
constexpr int la_chunk(bool bf16) { return bf16 ? 64 : 32; }   // positions of a chunk
constexpr int la_threads(int dvs) { return dvs / 16 * kWave; }

// waves of a SIMD that registers are kept for (LDS holds three workgroups of bf16's 64 x 64 outputs)
constexpr int la_waves(bool bf16, int dk, bool out) { return dk == 256 ? 2 : bf16 && dk == 64 && out ? 3 : 4; }

template <bool BF16, int DK, int DVS, bool OUT, bool VEC>
__global__ __launch_bounds__(la_threads(DVS), la_waves(BF16, DK, OUT)) void k_lattn_chunk(LattnCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    using Four = T __attribute__((ext_vector_type(4)));
    constexpr int C = la_chunk(BF16), KB = M::KB, E = M::E, NTH = la_threads(DVS), WAVES = NTH / kWave;
    constexpr int PK = DK + E, PV = DVS + E;                     // K's and V's LDS rows, 16 bytes longer
    constexpr int KT = DK / 16, CT = C / 16;                     // tiles of dk and of C
    constexpr int UK = C * DK / E / NTH, UV = C * DVS / E / NTH; // 16-byte units of a thread
    constexpr int PARTS = BF16 ? 2 : 1;                          // of an fp32 factor as an operand
    __shared__ __align__(16) T ks[C * PK], vs[C * PV], qs[OUT ? C * DK : 1], ps[OUT ? PARTS * C * C : 1];

    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    uint32_t l16 = (uint32_t)lane % 16, g = (uint32_t)lane / 16;
    const int slices = (a.dv + DVS - 1) / DVS, tasks = a.B * a.Hkv, shares = OUT ? slices * a.hsplit : slices;
    // the slices (and shares of query heads) of one segment read the same Q and K: eight workgroups apart, on one XCD and its L2
    const int unit = blockIdx.x / (8 * shares) * 8 + blockIdx.x % 8, share = blockIdx.x / 8 % shares, slice = share % slices;
    if (unit >= tasks * a.nseg) return;
    const int seg = unit / tasks, task = unit % tasks, b = task / a.Hkv, n = task % a.Hkv, col0 = slice * DVS;
    const int dk = a.dk, dv = a.dv;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool in = slot >= 0 && slot < a.n_slots;
    int len = a.lens ? a.lens[b] : a.L;
    len = in ? (len < 0 ? 0 : len > a.L ? a.L : len) : 0;
    const int chunks = (len + C - 1) / C, pad = chunks * C - len;
    const int c0 = seg * a.seg_chunks;
    int c1 = c0 + a.seg_chunks;
    if (c1 > chunks) c1 = chunks;
    if (!OUT && c1 >= chunks) return;   // a row's last segment hands nothing on
    const int per = OUT ? (a.G + a.hsplit - 1) / a.hsplit : 0, h0 = share / slices * per, h1 = h0 + per < a.G ? h0 + per : a.G;
    if (OUT && h0 >= h1) return;

    if (OUT) {   // o is zero past the row's end
        const int64_t z1 = seg == a.nseg - 1 ? a.L : (int64_t)(c0 + a.seg_chunks) * C < a.L ? (c0 + a.seg_chunks) * C : a.L;
        const int64_t z0 = len > c0 * C ? len : c0 * C;
        constexpr int Z = VEC ? E : 1, UNITS = DVS / Z;   // elements of a store, stores of a row
        const int col = col0 + tid % UNITS * Z;
        if (col < dv)
            for (int h = n * a.G + h0; h < n * a.G + h1; ++h)
                for (int64_t t = z0 + tid / UNITS; t < z1; t += NTH / UNITS) {
                    T* const p = static_cast<T*>(a.o.p) + b * a.o.row + t * a.o.pos + h * a.o.head + col;
                    if constexpr (VEC) *gmem(reinterpret_cast<Frag*>(p)) = Frag{};
                    else *gmem(p) = (T)0.f;
                }
        if (c0 >= chunks && !(seg == 0 && in && h0 == 0)) return;
    }

    // the lane's part of S: rows 16 kt + row0 + r of column scol
    const float ld = a.ld[n];
    V4 S[KT] = {};
    float* const sp = a.state && in ? a.state + (slot * a.Hkv + n) * dk * (int64_t)dv : nullptr;
    float* const wp = a.entries ? a.ws + ((int64_t)task * a.nseg + seg) * dk * dv : nullptr;
    const float* const from = !OUT ? nullptr : wp ? wp : a.fresh ? nullptr : sp;
    const bool full = dk == DK && col0 + DVS <= dv;   // no part of S lies outside
    // Some of the wave's columns are there; a wave without any leaves the matrix
    // cores to the others (38 -> 26 us, 12 heads of 192 x 32, fp32, 85 positions; in
    // slices of 64 columns the question costs more than it gives).
    const bool active = DVS <= 64 || col0 + 16 * wave < dv;
    // fp32's wide heads, whose products take most of the time, also leave out the
    // tiles beyond dk (us, 7 rows of 11096, 6 heads on 3, dk = 192 / 256, dv = 192: 1143 / 1396,
    // with all tiles 1343 / 1329; bf16, 3 of 31068, 10 on 5: 787 / 821 and 802 / 751).
    constexpr bool SHORT = !BF16 && DK > 128;
    if (from) {
        const int row0 = 4 * g, scol = col0 + 16 * wave + (int)l16;
        if (full) {
            const float* p = from + row0 * dv + scol;
#pragma unroll
            for (int i = 0; i < 4 * KT; ++i) S[i / 4][i % 4] = gmem(p)[(i / 4 * 16 + i % 4) * dv];
        } else if (scol < dv) {
#pragma unroll
            for (int i = 0; i < 4 * KT; ++i) {
                const int row = row0 + i / 4 * 16 + i % 4;
                if (row < dk) S[i / 4][i % 4] = gmem(from)[row * dv + scol];
            }
        }
    }

    // lam^i, and lam^{C-1-i}: the decay of a chunk's rows to its end
    __shared__ __align__(16) float lam[C + 1], to_end[C];
    for (int i = tid; i <= C; i += NTH) {
        lam[i] = decay_pow(ld, i);
        if (i < C) to_end[i] = decay_pow(ld, C - 1 - i);
    }
    const auto uniform = [](float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x))); };
    const float em1 = uniform(expm1f(C * ld)), em1_first = uniform(expm1f((C - pad) * ld));   // lam^n - 1

    // Staging: a thread has the same columns of rows RK (RV) apart.  Loads are
    // of valid places always (columns past the head's end and zero rows in
    // front repeat another one) and are blanked on their way to LDS.
    constexpr int RK = NTH * E / DK, RV = NTH * E / DVS;
    const int kcol = tid % (DK / E) * E, krow = tid / (DK / E), vcol = tid % (DVS / E) * E, vrow = tid / (DVS / E);
    const bool kin = kcol < dk, vin = col0 + vcol < dv;
    const int kleft = kin ? dk - kcol : 0, vleft = vin ? dv - col0 - vcol : 0;   // elements from there on
    const int klcol = kin ? kcol : 0, vlcol = vin ? vcol : 0;
    const T* const kp = static_cast<const T*>(a.k.p) + b * a.k.row + n * a.k.head;
    const T* const vp = static_cast<const T*>(a.v.p) + b * a.v.row + n * a.v.head + col0;
    const T* const qp = static_cast<const T*>(a.q.p) + b * a.q.row + ((int64_t)n * a.G + h0) * a.q.head;
    Frag fk[UK], fv[UV], fq[UK];
    // VEC: a chunk of rows spans less than 2^31 bytes, so that a place is a
    // wave's own base and a lane's 32-bit offset
    const auto fetch = [&](auto& f, const T* p, int64_t pos, int c, int row, int step, int col, int left) {
        constexpr int count = sizeof(f) / sizeof(f[0]);
        const int t0 = c * C - pad;
        int r[count];
#pragma unroll
        for (int i = 0; i < count; ++i) r[i] = row + i * step;
        if (t0 < 0) {   // (a zero row in front: the row's first position)
#pragma unroll
            for (int i = 0; i < count; ++i) r[i] = t0 + r[i] > 0 ? t0 + r[i] : 0;
        } else p += t0 * pos;
#pragma unroll
        for (int i = 0; i < count; ++i) {
            if constexpr (VEC) {
                const uint32_t off = (uint32_t)(r[i] * (int)pos + col) * sizeof(T);
                f[i] = *gmem(reinterpret_cast<const Frag*>(reinterpret_cast<const char*>(p) + off));
            } else f[i] = load_loose<BF16>(p + r[i] * pos + col, 0, left);
        }
    };
    const auto put = [&](T* to, int pitch, auto& f, int row, int step, int col, bool in, bool blank, int first) {
        constexpr int count = sizeof(f) / sizeof(f[0]);
        T* p = to + row * pitch + col;
        if (blank) {
#pragma unroll
            for (int i = 0; i < count; ++i)
                if (!in || row + i * step < first) f[i] = Frag{};
        }
#pragma unroll
        for (int i = 0; i < count; ++i) *smem_ptr(reinterpret_cast<Frag*>(p + i * step * pitch)) = f[i];
    };
    // Q and P: unit u of row r at u ^ r (rows of 8 units: u ^ r / 2), so that
    // 16 lanes with 16 rows meet every bank once whichever units they read
    const auto mixed = [](int units, uint32_t row, uint32_t u) { return (row * units + (u ^ (units == 8 ? row / 2 % 8 : row % 16))) * E; };
    // Q's rows, for whole 16-byte operand reads beside S's (whose lanes hold
    // rows 4 g .. 4 g + 3 of two tiles): each block of KB columns is stored in
    // the order 4 (g, tile) + r
    const auto put_q = [&](bool blank, int first) {
        {
#pragma unroll
            for (int i = 0; i < UK; ++i) {
                if (blank && (!kin || krow + i * RK < first)) fq[i] = Frag{};
                const int row = krow + i * RK, u = kcol / E;
                if constexpr (BF16) {
                    const int at = u / 4 * 4 + u % 2 * 2, half = u / 2 % 2 * 4;
                    *smem_ptr(reinterpret_cast<BF4*>(qs + mixed(DK / E, row, at) + half)) = __builtin_shufflevector(fq[i], fq[i], 0, 1, 2, 3);
                    *smem_ptr(reinterpret_cast<BF4*>(qs + mixed(DK / E, row, at + 1) + half)) = __builtin_shufflevector(fq[i], fq[i], 4, 5, 6, 7);
                } else *smem_ptr(reinterpret_cast<Frag*>(qs + mixed(DK / E, row, u))) = fq[i];
            }
        }
    };
    // 16 columns from col, as an operand over the KB positions from row t0
    const auto transposed = [&](const T* from, int pitch, int t0, int col) {
        Frag f;
        if constexpr (BF16) {
            // a 16-lane group reads 4 positions x 16 columns and gets them
            // transposed.  Positions 8 g + 2 e + h (element 4 h + e): two
            // apart, so that with rows of 4 banks more than a multiple of 64
            // the groups of a half wave meet no bank twice
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const T* p = from + (t0 + 8 * g + 2 * (l16 / 4) + h) * pitch + col + l16 % 4 * 4;
                const S4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FI_SHARED S4*)(p));
                const BF4 y = __builtin_bit_cast(BF4, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[4 * h + e] = y[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = smem_ptr(from)[(t0 + 4 * g + e) * pitch + col + l16];
        }
        return f;
    };
    // the operand in the order of Q's columns, from a row in its own
    const auto pair_frag = [&](const T* p) -> Frag {
        if constexpr (BF16) {
            const BF4 a = *smem_ptr(reinterpret_cast<const BF4*>(p)), b = *smem_ptr(reinterpret_cast<const BF4*>(p + 16));
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else return *smem_ptr(reinterpret_cast<const Frag*>(p));
    };
    const auto row_frag = [&](const T* p) { return *smem_ptr(reinterpret_cast<const Frag*>(p)); };

    if (c0 < c1) {
        fetch(fk, kp, a.k.pos, c0, krow, RK, klcol, kleft);
        fetch(fv, vp, a.v.pos, c0, vrow, RV, vlcol, vleft);
        if constexpr (OUT) fetch(fq, qp, a.q.pos, c0, krow, RK, klcol, kleft);
    }
    for (int c = c0; c < c1; ++c) {
        const int first = c == 0 ? pad : 0;   // zero rows in front
        const bool blank = first || !full;
        // the lane's place anew in every chunk: addresses that depend on it
        // are not all kept in registers around the loop
        asm volatile("" : "+v"(l16), "+v"(g));
        put(ks, PK, fk, krow, RK, kcol, kin, blank, first);
        put(vs, PV, fv, vrow, RV, vcol, vin, blank, first);
        if constexpr (OUT) put_q(blank, first);
        __syncthreads();
        // the next chunk's rows (the last one's again at the end: no branch,
        // so that nothing waits for them before their use)
        const int ahead = c + 1 < c1 ? c + 1 : c;
        // (K's rows beside V's where registers are short: of 128 columns they went to
        // scratch as soon as they came, 64K x 16 heads 446 us, 429 so; of 256 1% the other way)
        constexpr bool LATE = OUT && DK <= 128;
        if constexpr (!LATE) fetch(fk, kp, a.k.pos, ahead, krow, RK, klcol, kleft);
        if constexpr (!OUT) fetch(fv, vp, a.v.pos, ahead, vrow, RV, vlcol, vleft);
        if constexpr (OUT) {
            for (int h = h0; h < h1; ++h) {
                const bool last = h + 1 == h1;
                asm volatile("" : "+v"(l16), "+v"(g));
                // P^T, tiles of 16 keys x 16 queries, jt <= it, shared out among the waves
#pragma unroll
                for (int at = 0; at < CT * (CT + 1) / 2; at += WAVES) {
                    const int tile = at + wave;
                    if (tile >= CT * (CT + 1) / 2) break;
                    const int it = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, jt = tile - it * (it + 1) / 2;
                    const uint32_t krow_ = BF16 ? 8 * (l16 / 8) + 2 * (l16 % 4) + l16 / 4 % 2 : l16;
                    V4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int kb = 0; kb < DK / KB; ++kb) {
                        if (SHORT && kb * KB >= dk) break;
                        p = M::mma(pair_frag(ks + (16 * jt + krow_) * PK + kb * KB + 4 * g),
                                   row_frag(qs + mixed(DK / E, 16 * it + l16, kb * 4 + g)), p);
                    }
                    const auto to = [&](int tile, int part) {   // of four of the wave's 16 keys
                        return smem_ptr(reinterpret_cast<Four*>(ps + part * C * C + mixed(C / E, 16 * it + l16, (16 * tile + 4 * g) / E) + 4 * g % E));
                    };
                    const auto key = [&](int r) { return (int)(BF16 ? 8 * (g / 2) + 2 * r + g % 2 : 4 * g + r); };   // its place in its tile
                    if (it == jt) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int i = (int)l16 - key(r);
                            p[r] = (i >= 0 ? p[r] : 0.f) * lam[i >= 0 ? i : 0];
                        }
                        // the rest of the block of keys that the product below takes whole
                        if (BF16 && it % 2 == 0) *to(jt + 1, 0) = *to(jt + 1, 1) = Four{};
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) p[r] *= lam[16 * (it - jt) + (int)l16 - key(r)];
                    }
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        Four y;
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            y[r] = (T)p[r];
                            p[r] -= (float)y[r];
                        }
                        *to(jt, i) = y;
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                // O^T = E^T Q^T: columns are positions
                V4 O[CT] = {};
#pragma unroll
                for (int kb = 0; kb < DK / KB; ++kb) {
                    if (!active || (SHORT && kb * KB >= dk)) break;
                    Frag fs[PARTS];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        float x = S[kb * (KB / 16) + e / 4][e % 4];
#pragma unroll
                        for (int i = 0; i < PARTS; ++i) {
                            fs[i][e] = (T)x;
                            x -= (float)fs[i][e];
                        }
                    }
#pragma unroll
                    for (int it = 0; it < CT; ++it) {
                        const Frag q = row_frag(qs + mixed(DK / E, 16 * it + l16, kb * 4 + g));
#pragma unroll
                        for (int i = PARTS - 1; i >= 0; --i) O[it] = M::mma(fs[i], q, O[it]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                // (loads in three places: each waits for the address path otherwise)
                fetch(fq, qp + (last ? 0 : h + 1 - h0) * a.q.head, a.q.pos, last ? ahead : c, krow, RK, klcol, kleft);
                // lam^{i + 1}, counted from the row's first position in a first chunk
#pragma unroll
                for (int it = 0; it < CT; ++it) {
                    const int i = 16 * it + (int)l16 + 1 - first;
                    O[it] *= lam[i > 0 ? i : 0];
                }
                __syncthreads();
#pragma unroll
                for (int kb = 0; kb < C / KB; ++kb) {
                    if (!active) break;
                    const Frag v = transposed(vs, PV, kb * KB, 16 * wave);
#pragma unroll
                    for (int it = kb * KB / 16; it < CT; ++it)   // queries before every key of the block: nothing
#pragma unroll
                        for (int i = PARTS - 1; i >= 0; --i)
                            O[it] = M::mma(v, row_frag(ps + i * C * C + mixed(C / E, 16 * it + l16, kb * 4 + g)), O[it]);
                }
                __builtin_amdgcn_sched_barrier(0);
                T* const op = static_cast<T*>(a.o.p) + b * a.o.row + (n * a.G + h) * a.o.head + (int64_t)(c * C - pad) * a.o.pos + col0 + 16 * wave;
                const int left = dv - (col0 + 16 * wave + 4 * (int)g);
#pragma unroll
                for (int it = 0; it < CT; ++it) {
                    Four y;
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = (T)(a.scale * O[it][r]);
                    if (16 * it + (int)l16 >= first) {
                        if constexpr (VEC) {
                            const uint32_t off = (uint32_t)(l16 * (int)a.o.pos + 4 * g) * sizeof(T);
                            if (left > 0) *gmem(reinterpret_cast<Four*>(reinterpret_cast<char*>(op + 16 * it * a.o.pos) + off)) = y;
                        } else {
                            T* to = op + (16 * it + l16) * a.o.pos + 4 * g;
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (r < left) gmem(to)[r] = y[r];
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                if (!last) {
                    __syncthreads();
                    put_q(blank, first);
                    __syncthreads();
                }
            }
        }
        if constexpr (LATE) fetch(fk, kp, a.k.pos, ahead, krow, RK, klcol, kleft);
        if constexpr (OUT) fetch(fv, vp, a.v.pos, ahead, vrow, RV, vlcol, vleft);
        // S: its decay as S + (lam^C - 1) S (lam^C's rounding would add up
        // over the chunks of a long memory), then the chunk's own products
        const float d = c == 0 ? em1_first : em1;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[kt][r] = fmaf(d, S[kt][r], S[kt][r]);
#pragma unroll
        for (int kb = 0; kb < C / KB; ++kb) {
            if (!active) break;
            __builtin_amdgcn_sched_barrier(0);
            const Frag v = transposed(vs, PV, kb * KB, 16 * wave);
            float w[E];   // of the operand's positions
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                const V4 x = *smem_ptr(reinterpret_cast<const V4*>(to_end + kb * KB + E * g + e));
#pragma unroll
                for (int i = 0; i < 4; ++i) w[BF16 ? (e + i) / 2 + (i % 2) * 4 : i] = x[i];
            }
            if constexpr (BF16) {
                // V's decayed rows as the sum of three bf16 parts, each the top
                // 8 bits of what is left: exact, so that the state keeps fp32's precision
                uint32_t part[3][E / 2];
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    float x = (float)v[e] * w[e], y = (float)v[e + 1] * w[e + 1];
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
                        part[i][e / 2] = __builtin_amdgcn_perm(uy, ux, 0x07060302);   // the upper halves
                        x -= __uint_as_float(ux & 0xFFFF0000u);
                        y -= __uint_as_float(uy & 0xFFFF0000u);
                    }
                }
                const Frag hi = __builtin_bit_cast(Frag, part[0]), mid = __builtin_bit_cast(Frag, part[1]),
                           lo = __builtin_bit_cast(Frag, part[2]);
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    if (SHORT && kt % 4 == 0 && 16 * kt >= dk) break;
                    const Frag k = transposed(ks, PK, kb * KB, 16 * kt);
                    S[kt] = M::mma(k, hi, M::mma(k, mid, M::mma(k, lo, S[kt])));
                    if (kt % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
            } else {
                Frag x;
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = v[e] * w[e];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    if (SHORT && kt % 4 == 0 && 16 * kt >= dk) break;
                    S[kt] = M::mma(transposed(ks, PK, kb * KB, 16 * kt), x, S[kt]);
                }
            }
        }
        __syncthreads();
    }
    float* to = OUT ? (c1 == chunks && h0 == 0 ? sp : nullptr) : wp + (int64_t)dk * dv;
    if (!to) return;
    // the lane's place anew: nothing of the loads above is kept through the loop
    int row0 = 4 * g, scol = col0 + 16 * wave + (int)l16;
    asm volatile("" : "+v"(row0), "+v"(scol));
    if (full) {
        to += row0 * dv + scol;
#pragma unroll
        for (int i = 0; i < 4 * KT; ++i) gmem(to)[(i / 4 * 16 + i % 4) * dv] = S[i / 4][i % 4];
    } else if (scol < dv) {
#pragma unroll
        for (int i = 0; i < 4 * KT; ++i) {
            const int row = row0 + i / 4 * 16 + i % 4;
            if (row < dk) gmem(to)[row * dv + scol] = S[i / 4][i % 4];
        }
    }
}

// Entry states of a split row's segments, in place: ws[s + 1] holds the
// segment s's own products and becomes lam^{n_s} ws[s] + those; ws[0] = S_0.
template <bool BF16>
__global__ __launch_bounds__(256) void k_lattn_scan(LattnCall a) {
    constexpr int C = la_chunk(BF16);
    const int per = a.dk * a.dv, blocks = (per + 255) / 256;
    const int task = blockIdx.x / blocks, b = task / a.Hkv, n = task % a.Hkv;
    const int i = blockIdx.x % blocks * 256 + threadIdx.x;
    const int64_t slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.n_slots || i >= per) return;
    int len = a.lens ? a.lens[b] : a.L;
    len = len < 0 ? 0 : len > a.L ? a.L : len;
    const int chunks = (len + C - 1) / C, segs = (chunks + a.seg_chunks - 1) / a.seg_chunks;
    const float ld = a.ld[n];
    float* w = a.ws + (int64_t)task * a.nseg * per + i;
    float S = a.fresh || !a.state ? 0.f : a.state[(slot * a.Hkv + n) * per + i];
    w[0] = S;
    const float em1 = expm1f((float)(a.seg_chunks * C) * ld);
    float d = expm1f((float)(a.seg_chunks * C - (chunks * C - len)) * ld);   // the first segment is shorter
    // loads are asked for eight segments at a time: one at a time each waits for
    // memory (7.5 us where this takes 5.3, 32 heads of 64 x 64 in 16 segments)
    for (int s0 = 1; s0 < segs; s0 += 8) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = w[(int64_t)(s0 + j < segs ? s0 + j : segs - 1) * per];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (s0 + j >= segs) break;
            S = fmaf(d, S, S) + x[j];
            w[(int64_t)(s0 + j) * per] = S;
            d = em1;
        }
    }
}

namespace {

constexpr int kLaWorkgroups = 512;   // wanted of a launch: two for each CU (16 heads of 65536: 416 us, with 1024 447)
constexpr int kLaWhole = 4;          // chunks of a row that is not split

// Most segments of a row.  Each chunk of a segment takes its time twice (some 5 us
// in all), each segment its part of the scan (0.15 us): chunks per segment near
// the root of chunks / 32 (2 heads of 80 x 96, two rows of 2976, us with at least 4
// / 2 / 1 chunks a segment: 40 / 30 / 26; 2 heads of 96 x 96, one row of 16384, 4 / 1:
// 49 / 58).
int64_t chunks_each(int64_t chunks) {
    int64_t each = 1;
    while (32 * each * each < chunks) ++each;
    return each;
}
int64_t most_segments(int64_t chunks) { return chunks <= kLaWhole ? 1 : chunks / chunks_each(chunks); }

int slice_cols(int dk) { return dk <= 64 ? 64 : 128; }

// segments that a call of `tasks` rows and heads is split into
int segments(int64_t tasks, int slices, int chunks, int* seg_chunks) {
    int64_t n = kLaWorkgroups / (tasks * slices);
    if (n > most_segments(chunks)) n = most_segments(chunks);
    if (n < 1) n = 1;
    *seg_chunks = chunks ? (int)((chunks + n - 1) / n) : 1;
    return chunks ? (chunks + *seg_chunks - 1) / *seg_chunks : 1;
}

// workgroups that share out a group's query heads in a launch of so many without
int64_t head_shares(int64_t wgs) { return wgs < kLaWorkgroups ? kLaWorkgroups / (wgs > 0 ? wgs : 1) : 1; }

template <bool BF16, int DK, int DVS, bool VEC>
void chunk_launches(const LattnCall& c, hipStream_t st) {
    const int slices = (c.dv + DVS - 1) / DVS;
    const int64_t units = c.B * c.Hkv * c.nseg;
    const unsigned grid = (unsigned)((units + 7) / 8 * 8 * slices);
    if (c.nseg > 1) k_lattn_chunk<BF16, DK, DVS, false, VEC><<<grid, la_threads(DVS), 0, st>>>(c);
    if (c.entries)
        k_lattn_scan<BF16><<<(unsigned)(c.B * c.Hkv * ((c.dk * c.dv + 255) / 256)), 256, 0, st>>>(c);
    k_lattn_chunk<BF16, DK, DVS, true, VEC><<<grid * c.hsplit, la_threads(DVS), 0, st>>>(c);
}

template <bool BF16>
hipError_t chunk_dims(const LattnCall& c, hipStream_t st) {
    if (c.dk <= 64) c.vec ? chunk_launches<BF16, 64, 64, true>(c, st) : chunk_launches<BF16, 64, 64, false>(c, st);
    else if (c.dk <= 128) c.vec ? chunk_launches<BF16, 128, 128, true>(c, st) : chunk_launches<BF16, 128, 128, false>(c, st);
    else c.vec ? chunk_launches<BF16, 256, 128, true>(c, st) : chunk_launches<BF16, 256, 128, false>(c, st);
    return hipGetLastError();
}

}  // namespace

void plan_lattn(LattnCall& c) {
    const int cols = slice_cols(c.dk), slices = (c.dv + cols - 1) / cols, C = la_chunk(c.io_bf16);
    c.nseg = segments(c.B * c.Hkv, slices, (c.L + C - 1) / C, &c.seg_chunks);
    // A group's query heads go to workgroups of their own where the CUs are not
    // full without; each forms the state for itself, from the entry states' copy,
    // and the first writes it.  (A copy for this alone pays where every head gets
    // its own: 16 heads of 256 x 192 with 3 each, six given states, 16 positions: 33
    // us without, 70 with.)  32 heads on 8 of 128 x 128, one row of 512: 62 us
    // without, 32 with.
    const int64_t n = head_shares(c.B * c.Hkv * c.nseg * slices);
    c.hsplit = n >= c.G ? c.G : c.fresh || c.nseg > 1 ? (int)n : 1;
    c.entries = c.nseg > 1 || (c.hsplit > 1 && !c.fresh);
}

size_t lattn_ws_used(const LattnCall& c) { return c.entries ? (size_t)c.B * c.Hkv * c.nseg * c.dk * c.dv * sizeof(float) : 0; }

size_t lattn_ws_bytes(int64_t B, int64_t L, int H, int Hkv, int dk, int dv, int io_bf16) {
    const int C = la_chunk(io_bf16), cols = slice_cols(dk), slices = (dv + cols - 1) / cols;
    // most segments of any row: the longest's, or those of the longest with fewer chunks in each
    const int64_t chunks = (L + C - 1) / C, split = std::max(most_segments(chunks), 32 * (chunks_each(chunks) - 1));
    int64_t most = 0;   // states of any call: one of b rows has at most cap segments a row
    for (int64_t b = 1; b <= B && b * Hkv * slices <= kLaWorkgroups; ++b) {
        const int64_t cap = kLaWorkgroups / (b * Hkv * slices), n = std::min(cap, split);
        if ((n > 1 || (H > Hkv && head_shares(b * Hkv * slices) > 1)) && b * Hkv * n > most) most = b * Hkv * n;
    }
    return (size_t)most * dk * dv * sizeof(float);
}

hipError_t launch_lattn_chunk(LattnCall c, hipStream_t st) {
    plan_lattn(c);
    return c.io_bf16 ? chunk_dims<true>(c, st) : chunk_dims<false>(c, st);
}

}  // namespace fi
