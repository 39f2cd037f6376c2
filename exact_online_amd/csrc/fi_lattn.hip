// fi_lattn.hip -- linear attention with a decay per head (fi_lattn_*).
//
// Per row b, key/value head n and position t, lam = exp(ld[n]):
//     S[t] = lam S[t-1] + k[t] v[t]^T,   o[t][h] = scale S[t]^T q[t][h].
#include "fi_opdev.hpp"

namespace fi {

// ------------------------------------------------------------ recurrent form
// A workgroup holds dk x 32 of one (row, head)'s state in registers: thread
// (r, c) = (tid / 8, tid % 8) has the columns 4c .. 4c+3 of the slice and the
// rows r, r + 32, ...  Columns of S never meet, so slices need no exchange.
constexpr int kRecThreads = 256;
constexpr int kRecCols = 32;
constexpr int kRecRows = kRecThreads / (kRecCols / 4);   // rows in one sweep
constexpr int kRecHeads = 8;                             // query heads at a time

template <bool BF16, int RPT>
__global__ __launch_bounds__(kRecThreads) void k_lattn_rec(LattnCall a) {
    __shared__ float ks[kRecRows * RPT], vs[kRecCols], qs[kRecHeads][kRecRows * RPT];
    __shared__ float red[kRecThreads / kWave][kRecHeads][kRecCols];
    const int tid = threadIdx.x, c = tid % (kRecCols / 4), r = tid / (kRecCols / 4);
    const int slices = (a.dv + kRecCols - 1) / kRecCols;
    const int64_t b = blockIdx.x / slices / a.Hkv;
    const int n = blockIdx.x / slices % a.Hkv, col0 = blockIdx.x % slices * kRecCols;
    const int dk = a.dk, dv = a.dv, G = a.G;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool in = slot >= 0 && slot < a.n_slots;
    int len = a.lens ? a.lens[b] : a.L;
    len = in ? (len < 0 ? 0 : len > a.L ? a.L : len) : 0;
    const float em1 = expm1f(a.ld[n]);   // lam - 1
    float* const sp = a.state && in ? a.state + (slot * a.Hkv + n) * dk * (int64_t)dv : nullptr;

    float S[RPT][4];
    for (int i = 0; i < RPT; ++i)
        for (int j = 0; j < 4; ++j) {
            const int row = r + i * kRecRows, col = col0 + 4 * c + j;
            S[i][j] = !a.fresh && sp && row < dk && col < dv ? sp[row * (int64_t)dv + col] : 0.f;
        }
    for (int t = 0; t < len; ++t) {
        const int64_t kb = b * a.k.row + t * a.k.pos + n * a.k.head, vb = b * a.v.row + t * a.v.pos + n * a.v.head;
        for (int i = tid; i < kRecRows * RPT; i += kRecThreads) ks[i] = i < dk ? get_io<BF16>(a.k.p, kb + i) : 0.f;
        if (tid < kRecCols) vs[tid] = col0 + tid < dv ? get_io<BF16>(a.v.p, vb + col0 + tid) : 0.f;
        __syncthreads();
        // S + (lam - 1) S rather than lam S: the rounding of lam (up to 2^-25
        // of S a step, always to one side) would add up over long memories
        for (int i = 0; i < RPT; ++i)
            for (int j = 0; j < 4; ++j)
                S[i][j] = fmaf(ks[r + i * kRecRows], vs[4 * c + j], fmaf(em1, S[i][j], S[i][j]));
        for (int g0 = 0; g0 < G; g0 += kRecHeads) {
            const int gn = G - g0 < kRecHeads ? G - g0 : kRecHeads;
            __syncthreads();
            for (int i = tid; i < gn * kRecRows * RPT; i += kRecThreads) {
                const int g = i / (kRecRows * RPT), row = i % (kRecRows * RPT);
                qs[g][row] = row < dk ? get_io<BF16>(a.q.p, b * a.q.row + t * a.q.pos + (n * G + g0 + g) * a.q.head + row) : 0.f;
            }
            __syncthreads();
            for (int g = 0; g < gn; ++g)
                for (int j = 0; j < 4; ++j) {
                    float p = 0.f;
                    for (int i = 0; i < RPT; ++i) p = fmaf(qs[g][r + i * kRecRows], S[i][j], p);
                    for (int d = 8; d < kWave; d <<= 1) p += __shfl_xor(p, d);
                    if (tid % kWave < 8) red[tid / kWave][g][4 * c + j] = p;
                }
            __syncthreads();
            for (int i = tid; i < gn * kRecCols; i += kRecThreads) {
                const int g = i / kRecCols, col = i % kRecCols;
                const float o = red[0][g][col] + red[1][g][col] + red[2][g][col] + red[3][g][col];
                if (col0 + col < dv)
                    put_io<BF16>(a.o.p, b * a.o.row + t * a.o.pos + (n * G + g0 + g) * a.o.head + col0 + col, a.scale * o);
            }
        }
        __syncthreads();
    }
    for (int64_t i = (int64_t)len * G * kRecCols + tid; i < (int64_t)a.L * G * kRecCols; i += kRecThreads) {
        const int col = i % kRecCols, g = i / kRecCols % G, t = i / kRecCols / G;
        if (col0 + col < dv) put_io<BF16>(a.o.p, b * a.o.row + t * a.o.pos + (n * G + g) * a.o.head + col0 + col, 0.f);
    }
    if (sp)
        for (int i = 0; i < RPT; ++i)
            for (int j = 0; j < 4; ++j) {
                const int row = r + i * kRecRows, col = col0 + 4 * c + j;
                if (row < dk && col < dv) sp[row * (int64_t)dv + col] = S[i][j];
            }
}

hipError_t launch_lattn_rec(const LattnCall& c, hipStream_t st) {
    const bool small = c.dk <= 4 * kRecRows;
    const dim3 grid((unsigned)((c.dv + kRecCols - 1) / kRecCols * c.Hkv * c.B));   // B Hkv <= kLattnMaxRows
    if (c.io_bf16) {
        if (small) k_lattn_rec<true, 4><<<grid, kRecThreads, 0, st>>>(c);
        else k_lattn_rec<true, 8><<<grid, kRecThreads, 0, st>>>(c);
    } else {
        if (small) k_lattn_rec<false, 4><<<grid, kRecThreads, 0, st>>>(c);
        else k_lattn_rec<false, 8><<<grid, kRecThreads, 0, st>>>(c);
    }
    return hipGetLastError();
}

// ------------------------------------------------------------ chunked form
// A workgroup of four waves takes a segment of positions of one (row, head)
// and a slice of DVS columns of S, chunk by chunk.  With Q, K, V a chunk's
// rows, E the state before it and i, j < C:
//     O = scale (diag(lam^{i+1}) Q E + P V),  P[i][j] = lam^{i-j} q_i . k_j, j <= i
//     S = lam^C E + K^T diag(lam^{C-1-j}) V
// A row's first chunk is filled from the back (zero rows in front), so that
// every later one is whole and ends on the row's last position.
constexpr int kLaThreads = 256;
constexpr int la_chunk(bool bf16) { return bf16 ? 64 : 32; }   // positions of a chunk


// 16 bytes of a head's row: elements c .. c + E - 1 below d, zero elsewhere
template <bool BF16>
__device__ __forceinline__ typename Mm<BF16>::Frag load_unit(const void* p, int64_t at, int c, int d, bool vec) {
    using M = Mm<BF16>;
    typename M::Frag u = {};
    const typename M::T* q = static_cast<const typename M::T*>(p) + at + c;
    if (vec) {
        if (c < d) u = *gmem(reinterpret_cast<const typename M::Frag*>(q));
    } else {
#pragma unroll
        for (int e = 0; e < M::E; ++e)
            if (c + e < d) u[e] = gmem(q)[e];
    }
    return u;
}

template <bool BF16, int DK, int DVS, bool OUT>
__global__ __launch_bounds__(kLaThreads, 2) void k_lattn_chunk(LattnCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    constexpr int C = la_chunk(BF16), KB = M::KB, E = M::E;
    constexpr int PK = DK + E, PV = DVS + E, PP = C + E;   // LDS rows, 16 bytes longer
    constexpr int NT = DVS / 64, KT = DK / 16, CT = C / 16;               // column tiles of a wave; tiles of dk; of C
    constexpr int UK = C * DK / E / kLaThreads, UV = C * DVS / E / kLaThreads;   // 16-byte units per thread
    __shared__ __align__(16) T ks[C * PK], vs[C * PV], qs[OUT ? C * PK : 1], ps[OUT ? C * PP : 1];

    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, l16 = lane % 16, g = lane / 16;
    const int slices = (a.dv + DVS - 1) / DVS, tasks = a.B * a.Hkv;
    // the slices of one segment read the same Q and K: eight workgroups apart, on one XCD and its L2
    const int unit = blockIdx.x / (8 * slices) * 8 + blockIdx.x % 8, slice = blockIdx.x / 8 % slices;
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

    if (OUT) {   // o is zero past the row's end
        const int64_t z1 = seg == a.nseg - 1 ? a.L : (int64_t)(c0 + a.seg_chunks) * C < a.L ? (c0 + a.seg_chunks) * C : a.L;
        const int64_t z0 = len > c0 * C ? len : c0 * C;
        for (int64_t i = z0 * a.G * DVS + tid; i < z1 * a.G * DVS; i += kLaThreads) {
            const int col = col0 + i % DVS, h = n * a.G + i / DVS % a.G;
            if (col < dv) put_io<BF16>(a.o.p, b * a.o.row + i / DVS / a.G * a.o.pos + h * a.o.head + col, 0.f);
        }
        if (c0 >= chunks && !(seg == 0 && in)) return;
    }

    const float ld = a.ld[n];
    V4 S[KT][NT];
    // thread's part of S: rows 16 kt + 4 g + r, columns col0 + 16 (wave NT + nt) + l16
    float* const sp = a.state && in ? a.state + (slot * a.Hkv + n) * dk * (int64_t)dv : nullptr;
    float* const wp = a.nseg > 1 ? a.ws + ((int64_t)task * a.nseg + seg) * dk * dv : nullptr;
    const float* const from = !OUT ? nullptr : wp ? wp : a.fresh ? nullptr : sp;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * kt + 4 * g + r, col = col0 + 16 * (wave * NT + nt) + l16;
                S[kt][nt][r] = from && row < dk && col < dv ? from[row * dv + col] : 0.f;
            }

    // decays: of a chunk's rows to its end (per operand element), from its
    // start, and between positions of one tile and of tiles apart
    const float em1 = expm1f(C * ld), lamKB = decay_pow(ld, KB), lam16 = decay_pow(ld, 16);
    float to_end[E], near[4], apart[4];
#pragma unroll
    for (int e = 0; e < E; ++e) to_end[e] = decay_pow(ld, KB - 1 - (BF16 ? 8 * g + 2 * (e % 4) + e / 4 : 4 * g + e));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int j = BF16 ? 8 * (g / 2) + 2 * r + g % 2 : 4 * g + r;   // the key's place in its tile
        near[r] = l16 >= j ? decay_pow(ld, l16 - j) : 0.f;
        apart[r] = decay_pow(ld, 16 + l16 - j);
    }
    const float from_start = decay_pow(ld, l16 + 1);

    Frag fk[UK], fv[UV], fq[UK];
    const auto load_kv = [&](int c) {
        const int t0 = c * C - pad;
#pragma unroll
        for (int i = 0; i < UK; ++i) {
            const int u = tid + i * kLaThreads, t = t0 + u / (DK / E), e = u % (DK / E) * E;
            fk[i] = t >= 0 ? load_unit<BF16>(a.k.p, b * a.k.row + t * a.k.pos + n * a.k.head, e, dk, a.vec) : Frag{};
        }
#pragma unroll
        for (int i = 0; i < UV; ++i) {
            const int u = tid + i * kLaThreads, t = t0 + u / (DVS / E), e = u % (DVS / E) * E;
            fv[i] = t >= 0 ? load_unit<BF16>(a.v.p, b * a.v.row + t * a.v.pos + n * a.v.head, col0 + e, dv, a.vec) : Frag{};
        }
    };
    const auto load_q = [&](int c, int h) {
        const int t0 = c * C - pad;
#pragma unroll
        for (int i = 0; i < UK; ++i) {
            const int u = tid + i * kLaThreads, t = t0 + u / (DK / E), e = u % (DK / E) * E;
            fq[i] = t >= 0 ? load_unit<BF16>(a.q.p, b * a.q.row + t * a.q.pos + (n * a.G + h) * a.q.head, e, dk, a.vec) : Frag{};
        }
    };
    const auto put = [&](T* to, int pitch, int per_row, int u, Frag f) {
        *smem_ptr(reinterpret_cast<Frag*>(to + u / per_row * pitch + u % per_row * E)) = f;
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
            for (int e = 0; e < 4; ++e) f[e] = from[(t0 + 4 * g + e) * pitch + col + l16];
        }
        return f;
    };
    const auto row_frag = [&](const T* p) { return *smem_ptr(reinterpret_cast<const Frag*>(p)); };

    if (c0 < c1) {
        load_kv(c0);
        if (OUT) load_q(c0, 0);
    }
    for (int c = c0; c < c1; ++c) {
        const int first = c == 0 ? pad : 0;   // zero rows in front
#pragma unroll
        for (int i = 0; i < UK; ++i) put(ks, PK, DK / E, tid + i * kLaThreads, fk[i]);
#pragma unroll
        for (int i = 0; i < UV; ++i) put(vs, PV, DVS / E, tid + i * kLaThreads, fv[i]);
        if constexpr (OUT) {
            for (int h = 0; h < a.G; ++h) {
#pragma unroll
                for (int i = 0; i < UK; ++i) put(qs, PK, DK / E, tid + i * kLaThreads, fq[i]);
                __syncthreads();
                if (h == 0 && c + 1 < c1) load_kv(c + 1);
                if (h + 1 < a.G) load_q(c, h + 1);
                else if (c + 1 < c1) load_q(c + 1, 0);
                // P^T of the wave's queries: tile jt of keys x its 16 queries
                if (wave < CT) {
                    Frag fq16[DK / KB];
#pragma unroll
                    for (int kb = 0; kb < DK / KB; ++kb) fq16[kb] = row_frag(qs + (16 * wave + l16) * PK + kb * KB + g * E);
                    const int krow = BF16 ? 8 * (l16 / 8) + 2 * (l16 % 4) + l16 / 4 % 2 : l16;
                    float far = 1.f;
                    for (int jt = wave; jt >= 0; --jt) {
                        V4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int kb = 0; kb < DK / KB; ++kb)
                            p = M::mma(row_frag(ks + (16 * jt + krow) * PK + kb * KB + g * E), fq16[kb], p);
                        if (jt == wave) {
#pragma unroll
                            for (int r = 0; r < 4; ++r) p[r] = near[r] == 0.f ? 0.f : p[r] * near[r];
                        } else {
#pragma unroll
                            for (int r = 0; r < 4; ++r) p[r] *= apart[r] * far;
                            far *= lam16;
                        }
                        T* to = ps + (16 * wave + l16) * PP + 16 * jt + 4 * g;
                        if constexpr (BF16) {
                            BF4 y;
#pragma unroll
                            for (int r = 0; r < 4; ++r) y[r] = (BF)p[r];
                            *smem_ptr(reinterpret_cast<BF4*>(to)) = y;
                        } else *smem_ptr(reinterpret_cast<V4*>(to)) = p;
                    }
                    // the rest of the key block that the product below takes whole
                    if (BF16 && wave % 2 == 0) *smem_ptr(reinterpret_cast<BF4*>(ps + (16 * wave + l16) * PP + 16 * (wave + 1) + 4 * g)) = BF4{};
                }
                // O^T = E^T Q^T: columns are positions
                V4 O[NT][CT] = {};
#pragma unroll
                for (int kb = 0; kb < DK / KB; ++kb) {
                    Frag fs[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < E; ++e) fs[nt][e] = (T)S[kb * (KB / 16) + e / 4][nt][e % 4];
#pragma unroll
                    for (int it = 0; it < CT; ++it) {
                        const T* p = qs + (16 * it + l16) * PK + kb * KB + 4 * g;
                        Frag f;
                        if constexpr (BF16) {
                            const BF4 lo = *smem_ptr(reinterpret_cast<const BF4*>(p)), hi = *smem_ptr(reinterpret_cast<const BF4*>(p + 16));
                            f = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                        } else f = row_frag(p);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) O[nt][it] = M::mma(fs[nt], f, O[nt][it]);
                    }
                }
                float w = first ? 1.f : from_start;
#pragma unroll
                for (int it = 0; it < CT; ++it) {
                    // lam^{i + 1}, counted from the row's first position in a first chunk
                    const int i = 16 * it + l16 + 1 - first;
                    const float f = first ? decay_pow(ld, i > 0 ? i : 0) : w;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) O[nt][it] *= f;
                    w *= lam16;
                }
                __syncthreads();
#pragma unroll
                for (int kb = 0; kb < C / KB; ++kb) {
                    Frag v[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) v[nt] = transposed(vs, PV, kb * KB, 16 * (wave * NT + nt));
#pragma unroll
                    for (int it = 0; it < CT; ++it) {
                        if (16 * it + 15 < kb * KB) continue;   // keys after every query
                        const Frag p = row_frag(ps + (16 * it + l16) * PP + kb * KB + g * E);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) O[nt][it] = M::mma(v[nt], p, O[nt][it]);
                    }
                }
                const int64_t ob = b * a.o.row + (n * a.G + h) * a.o.head;
#pragma unroll
                for (int it = 0; it < CT; ++it) {
                    const int t = c * C - pad + 16 * it + l16;
                    if (t < 0) continue;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int col = col0 + 16 * (wave * NT + nt) + 4 * g;
                        if (col >= dv) continue;
                        T* to = static_cast<T*>(a.o.p) + ob + t * a.o.pos + col;
                        using Four = T __attribute__((ext_vector_type(4)));
                        Four y;
#pragma unroll
                        for (int r = 0; r < 4; ++r) y[r] = (T)(a.scale * O[nt][it][r]);
                        if (a.vec) *gmem(reinterpret_cast<Four*>(to)) = y;
                        else
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (col + r < dv) gmem(to)[r] = y[r];
                    }
                }
                if (h + 1 < a.G) __syncthreads();
            }
        } else {
            __syncthreads();
            if (c + 1 < c1) load_kv(c + 1);
        }
        // S: its decay as S + (lam^C - 1) S (lam^C's rounding would add up
        // over the chunks of a long memory), then the chunk's own products
        const float d = first ? expm1f((C - first) * ld) : em1;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[kt][nt][r] = fmaf(d, S[kt][nt][r], S[kt][nt][r]);
        float far = 1.f;
#pragma unroll
        for (int kb = C / KB - 1; kb >= 0; --kb) {
            if constexpr (BF16) {
                // V's decayed rows as a sum of three bf16 parts (24 bits): the state keeps fp32's precision
                Frag hi[NT], mid[NT], lo[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const Frag v = transposed(vs, PV, kb * KB, 16 * (wave * NT + nt));
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float x = (float)v[e] * (to_end[e] * far);
                        hi[nt][e] = (BF)x;
                        const float y = x - (float)hi[nt][e];
                        mid[nt][e] = (BF)y;
                        lo[nt][e] = (BF)(y - (float)mid[nt][e]);
                    }
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const Frag k = transposed(ks, PK, kb * KB, 16 * kt);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        S[kt][nt] = M::mma(k, hi[nt], M::mma(k, mid[nt], M::mma(k, lo[nt], S[kt][nt])));
                }
            } else {
                Frag v[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    v[nt] = transposed(vs, PV, kb * KB, 16 * (wave * NT + nt));
#pragma unroll
                    for (int e = 0; e < E; ++e) v[nt][e] *= to_end[e] * far;
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const Frag k = transposed(ks, PK, kb * KB, 16 * kt);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) S[kt][nt] = M::mma(k, v[nt], S[kt][nt]);
                }
            }
            far *= lamKB;
        }
        __syncthreads();
    }
    float* to = OUT ? (c1 == chunks ? sp : nullptr) : wp + (int64_t)dk * dv;
    if (to)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * kt + 4 * g + r, col = col0 + 16 * (wave * NT + nt) + l16;
                    if (row < dk && col < dv) to[row * dv + col] = S[kt][nt][r];
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
    for (int s = 1; s < segs; ++s) {
        S = fmaf(d, S, S) + w[(int64_t)s * per];
        w[(int64_t)s * per] = S;
        d = em1;
    }
}

namespace {

constexpr int kLaWorkgroups = 512;   // wanted of a launch: two for each CU
constexpr int kLaMinChunks = 8;      // of a segment

int slice_cols(int dk) { return dk > 64 && dk <= 128 ? 128 : 64; }

// segments that a call of `tasks` rows and heads is split into
int segments(int64_t tasks, int slices, int chunks, int* seg_chunks) {
    int64_t n = kLaWorkgroups / (tasks * slices);
    if (n > chunks / kLaMinChunks) n = chunks / kLaMinChunks;
    if (n < 1) n = 1;
    *seg_chunks = (int)((chunks + n - 1) / n);
    return chunks ? (chunks + *seg_chunks - 1) / *seg_chunks : 1;
}

template <bool BF16, int DK, int DVS>
void chunk_launches(const LattnCall& c, hipStream_t st) {
    const int slices = (c.dv + DVS - 1) / DVS;
    const int64_t units = c.B * c.Hkv * c.nseg;
    const unsigned grid = (unsigned)((units + 7) / 8 * 8 * slices);
    if (c.nseg > 1) {
        k_lattn_chunk<BF16, DK, DVS, false><<<grid, kLaThreads, 0, st>>>(c);
        k_lattn_scan<BF16><<<(unsigned)(c.B * c.Hkv * ((c.dk * c.dv + 255) / 256)), 256, 0, st>>>(c);
    }
    k_lattn_chunk<BF16, DK, DVS, true><<<grid, kLaThreads, 0, st>>>(c);
}

template <bool BF16>
hipError_t chunk_dims(LattnCall& c, hipStream_t st) {
    const int cols = slice_cols(c.dk);
    c.nseg = segments(c.B * c.Hkv, (c.dv + cols - 1) / cols, (c.L + la_chunk(BF16) - 1) / la_chunk(BF16), &c.seg_chunks);
    if (c.dk <= 64) chunk_launches<BF16, 64, 64>(c, st);
    else if (c.dk <= 128) chunk_launches<BF16, 128, 128>(c, st);
    else chunk_launches<BF16, 256, 64>(c, st);
    return hipGetLastError();
}

}  // namespace

size_t lattn_ws_bytes(int64_t B, int64_t L, int Hkv, int dk, int dv, int io_bf16) {
    const int C = la_chunk(io_bf16), cols = slice_cols(dk), slices = (dv + cols - 1) / cols;
    int64_t most = 0;   // states of any call's segments; a call of n rows is split into at most kLaWorkgroups / n
    for (int64_t b = 1; b <= B && b * Hkv * slices <= kLaWorkgroups; ++b) {
        int sc;
        // a shorter call has no more segments than its chunks give
        int64_t n = segments(b * Hkv, slices, (int)((L + C - 1) / C), &sc);
        const int64_t cap = kLaWorkgroups / (b * Hkv * slices);
        if (n > 1 || L >= 2 * kLaMinChunks * C) n = cap < L / (kLaMinChunks * C) + 1 ? cap : L / (kLaMinChunks * C) + 1;
        if (n > 1 && b * Hkv * n > most) most = b * Hkv * n;
    }
    return (size_t)most * dk * dv * sizeof(float);
}

hipError_t launch_lattn_chunk(LattnCall c, hipStream_t st) {
    return c.io_bf16 ? chunk_dims<true>(c, st) : chunk_dims<false>(c, st);
}

}  // namespace fi
