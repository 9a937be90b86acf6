// experts.hip -- products of the expert-grouped rows with the experts' weights
// on gfx950: ep_expert_matmul, ep_expert_swiglu and ep_expert_wgrad.
//
// Rows i of expert e are [expert_offsets[e], expert_offsets[e+1]).
//   matmul  y[i][n]  = sum_k x[i][k] W[e][n][k]   (or W[e][k][n])
//   swiglu  g = x W13[e][0:F]^T, u = x W13[e][F:2F]^T, act = silu(g) u
//   wgrad   dW[e][n][k] = sum_{i of e} dy[i][n] x[i][k]
#include <algorithm>

#include "ep_internal.h"
#include "ep_mfma.h"

namespace ep {
namespace {

constexpr int kThreads = 512;   // 8 waves, two per SIMD
constexpr int kTileN = 256;     // columns of a tile
constexpr int kStep = 64;       // contracted indices per step
constexpr int kFullRows = 256;  // rows of a full tile
constexpr int kPart = 32768;    // LDS bytes of one operand's step (256 x 64 bf16)
constexpr int kRingB = 2 * kPart;  // two steps of the first operand, then three of the second
constexpr int kLdsBytes = 5 * kPart;

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(EP_LDS_PTR(const char))p;
}

// ---- Operand tiles in LDS ---------------------------------------------------
//
// "Rows" layout: ROWS rows of 64 contracted values (128 bytes, eight 16-byte
// chunks). Chunk c of row r lies at chunk c ^ ((r >> 1) & 7), which a wave's
// 16-byte reads pass without bank conflicts.
//
// "Columns" layout: 64 contracted rows of 256 values (512 bytes, sixteen
// 32-byte blocks). Block b of row k lies at block b ^ f(k), f(k) = (k & 3) |
// ((k >> 3) & 3) << 2: the 16 rows that a wave's transposing read touches then
// cover the banks evenly.
//
// Steps of 64 rather than 32 indices, so that every copy takes whole 128-byte
// lines: with 64-byte pieces a tile's copies alone filled the L2's requests
// (1060 against TFLOP/s at 32 experts of 1,024 x 7168 x 4096).

// An operand that needs no work between its copy and its reads.
struct NoStaging {
    __device__ __forceinline__ void stage(char*) {}
};

// A tile operand whose contracted index is contiguous in memory.
template <int ROWS>
struct RowsLoader : NoStaging {
    static constexpr int kLoads = ROWS / 64;
    const char* p;
    uint32_t bytes;
    uint32_t off[kLoads];
    int k;         // this lane's first contracted index within a step
    u32x4 d;       // descriptor of the step under way
    uint32_t far;  // added to the offsets: kBufFar where the step is past the end

    // row(r): byte offset of tile row r from p.
    template <class RowOff>
    __device__ __forceinline__ void init(const void* base, uint32_t n_bytes, RowOff row) {
        p = static_cast<const char*>(base);
        bytes = n_bytes;
        const int lane = lane_id(), wave = wave_in_block();
        const int r = wave * 8 + (lane >> 3);
        const int chunk = (lane & 7) ^ ((r >> 1) & 7);
        k = chunk * 8;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t o = row(j * 64 + r);
            off[j] = o == kBufOutside ? o : o + chunk * 16;
        }
    }
    // Turns to the step whose first index is k0 of k_dim (zeros past k_dim).
    __device__ __forceinline__ void begin(int k0, int k_dim) {
        d = buf_desc(p + (int64_t)k0 * 2, k0 < k_dim ? bytes - (uint32_t)k0 * 2 : 0u);
        far = k0 + k < k_dim ? 0u : kBufFar;
    }
    // Requests part j of kLoads of that step into LDS.
    __device__ __forceinline__ void copy(int j, uint32_t lds) {
        copy16_to_lds(d, off[j] + far, lds + (j * 64 + uniform_wave() * 8) * 128);
    }
};

// A tile operand whose 256 columns are contiguous in memory (one contracted
// index per memory row of ld values).
struct ColsLoader : NoStaging {
    static constexpr int kLoads = 4;
    const char* p;
    int64_t ld_bytes;
    uint32_t col_bytes;  // bytes of a row before the tile's first column
    uint32_t off[kLoads];
    u32x4 d;

    __device__ __forceinline__ void init(const void* base, int64_t ld, int col0) {
        p = static_cast<const char*>(base) + (int64_t)col0 * 2;
        ld_bytes = ld * 2;
        col_bytes = col0 * 2;
        const int lane = lane_id(), wave = wave_in_block();
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int r = j * 16 + wave * 2 + (lane >> 5);
            const int f = (r & 3) | (((r >> 3) & 3) << 2);
            const int block = ((lane & 31) >> 1) ^ f;
            off[j] = (uint32_t)(r * ld_bytes) + block * 32 + (lane & 1) * 16;
        }
    }
    __device__ __forceinline__ void begin(int k0, int k_dim) {
        const int rows = min(k_dim - k0, kStep);
        d = buf_desc(p + (int64_t)k0 * ld_bytes, rows > 0 ? (uint32_t)(rows * ld_bytes) - col_bytes : 0u);
    }
    __device__ __forceinline__ void copy(int j, uint32_t lds) {
        copy16_to_lds(d, off[j], lds + (j * 16 + uniform_wave() * 2) * 512);
    }
};

// 16 x 32 fragments of the step at lds: sub-tile s (16 rows or columns), half
// `half` of the contracted indices.
struct RowsReader {
    static constexpr int kReads = 1;  // LDS instructions per fragment
    uint32_t base[2];
    __device__ __forceinline__ void init(int first_sub) {
        const int i = lane_id() & 15, q = lane_id() >> 4;
        const uint32_t row = (first_sub * 16 + i) * 128;
        base[0] = row + ((q ^ (i >> 1)) * 16);
        base[1] = row + (((q + 4) ^ (i >> 1)) * 16);
    }
    __device__ __forceinline__ bf16x8 read(const char* lds, int s, int half) const {
        return *reinterpret_cast<const bf16x8*>(lds + base[half] + s * 2048);
    }
};
template <int SUBS>
struct ColsReader {
    static constexpr int kReads = 2;
    uint32_t base[SUBS];
    __device__ __forceinline__ void init(int first_sub) {
        const int i = lane_id() & 15, q = lane_id() >> 4;
        const int f = (i >> 2) | (q << 2);
#pragma unroll
        for (int s = 0; s < SUBS; ++s)
            base[s] = (q * 8 + (i >> 2)) * 512 + (((first_sub + s) ^ f) << 5) + (i & 3) * 8;
    }
    // Each 16-lane group reads 4 contracted rows of 16 values and receives
    // them transposed: lane i gets the 4 rows' values of column i.
    __device__ __forceinline__ bf16x8 read(const char* lds, int s, int half) const {
        const char* p = lds + base[s] + half * 16384;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((EP_LDS_PTR(s16x4))p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((EP_LDS_PTR(s16x4))(p + 2048));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, v);
    }
};

template <int MS, int NS>
struct Fragments {
    bf16x8 a[MS], b[NS];
};
// The fragments are wanted on the loop's way out too: without this the
// compiler moves their reads past the exit test, behind the matrix instructions
// that they should run beside.
template <int MS, int NS>
__device__ __forceinline__ void keep(const Fragments<MS, NS>& f) {
#pragma unroll
    for (int i = 0; i < MS; ++i) asm volatile("" ::"v"(f.a[i]));
#pragma unroll
    for (int i = 0; i < NS; ++i) asm volatile("" ::"v"(f.b[i]));
}

// One half step: multiplies the fragments `cur` while the fragments `next` are
// read from (la_lds, lb_lds, half), in MS groups of NS matrix instructions, each
// behind its share of the reads (all within the first GROUPS groups) and one
// of the copies: copies issued in one go would stand in the waves' way until
// the memory pipeline has taken them all (16 clocks each).
template <int MS, int NS, int GROUPS, class RA, class RB, class Copies>
__device__ __forceinline__ void half_step(const RA& ra, const RB& rb, const char* a_lds, const char* b_lds, int half,
                                          const Fragments<MS, NS>& cur, Fragments<MS, NS>& next,
                                          f32x4 (&acc)[MS][NS], Copies copies) {
    constexpr int R = MS + NS;
#pragma unroll
    for (int g = 0; g < MS; ++g) {
#pragma unroll
        for (int r = g * R / GROUPS; r < (g + 1) * R / GROUPS && r < R; ++r) {
            if (r < NS)
                next.b[r] = rb.read(b_lds, r, half);
            else
                next.a[r - NS] = ra.read(a_lds, r - NS, half);
        }
        copies(g);
#pragma unroll
        for (int n = 0; n < NS; ++n) acc[g][n] = mfma_bf16(cur.b[n], cur.a[g], acc[g][n]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// One workgroup's product: acc[mi][ni] += rows sub-tile mi times columns
// sub-tile ni over k_dim contracted indices. Each half of a step is multiplied
// from registers while the fragments of the next half are read from LDS, with
// one barrier per step. All of the LDS holds steps: two of the first operand,
// three of the second. In the first half of step s the copies of the second
// operand's step s + 2 are issued (into the slot of step s - 1), in the second
// half those of the first operand's (into the slot of step s, whose last
// fragments have then been read), so copies are spread over the whole step
// and have between one and two steps' time to arrive.
template <int MS, int NS, class LA, class LB, class RA, class RB>
__device__ __forceinline__ void multiply(LA& la, LB& lb, const RA& ra, const RB& rb, int k_dim, char* lds,
                                         f32x4 (&acc)[MS][NS]) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_address(lds));
    const int steps = (k_dim + kStep - 1) / kStep;
    if (steps > 0) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            la.begin(s * kStep, k_dim);
            lb.begin(s * kStep, k_dim);
            for (int c = 0; c < LA::kLoads; ++c) la.copy(c, at + s * kPart);
            for (int c = 0; c < LB::kLoads; ++c) lb.copy(c, at + kRingB + s * kPart);
            lb.stage(lds + kRingB + s * kPart);
        }
        Fragments<MS, NS> f[2];
        wait_copies<LA::kLoads + LB::kLoads>();
        barrier_only();
#pragma unroll
        for (int i = 0; i < NS; ++i) f[0].b[i] = rb.read(lds + kRingB, i, 0);
#pragma unroll
        for (int i = 0; i < MS; ++i) f[0].a[i] = ra.read(lds, i, 0);
        int b_now = kRingB, b_next = kRingB + kPart, b_free = kRingB + 2 * kPart;
        for (int s = 0; s < steps; s += 2) {
#pragma unroll
            for (int slot = 0; slot < 2; ++slot) {
                if (slot && s + 1 >= steps) break;
                lb.begin((s + slot + 2) * kStep, k_dim);
                half_step<MS, NS, MS>(ra, rb, lds + slot * kPart, lds + b_now, 1, f[0], f[1], acc, [&](int g) {
#pragma unroll
                    for (int c = g * LB::kLoads / MS; c < (g + 1) * LB::kLoads / MS; ++c) lb.copy(c, at + b_free);
                });
                wait_copies<LB::kLoads>();
                barrier_only();
                la.begin((s + slot + 2) * kStep, k_dim);
                half_step<MS, NS, MS>(ra, rb, lds + (slot ^ 1) * kPart, lds + b_next, 0, f[1], f[0], acc, [&](int g) {
#pragma unroll
                    for (int c = g * LA::kLoads / MS; c < (g + 1) * LA::kLoads / MS; ++c)
                        la.copy(c, at + slot * kPart);
                });
                lb.stage(lds + b_free);
                const int b = b_now;
                b_now = b_next, b_next = b_free, b_free = b;
            }
        }
        keep(f[0]);
        wait_copies<0>();  // none may land after the workgroup has left its LDS
    }
    settle(acc);
    barrier_only();  // the caller may use the slots again
}

// ---- Tiles of ragged experts ------------------------------------------------

struct Tile {
    int expert;
    int row0;   // first row of the tile
    int rows;   // rows of the tile that exist
    int n;      // column tile
    int shape;  // row capacity of the tile: 256 (full), else the tail's
};

// Finds this workgroup's tile; false if there is none. Every expert has
// floor(m / 256) full tiles and one tail of m % 256 rows, each times `n_tiles`.
// Full tiles come first (tails fill the gaps at the end). Workgroups go to the
// 8 XCDs in turn, so each XCD takes a contiguous run of tiles: within an
// expert the row tiles of one column tile follow each other, and the tiles that
// an XCD holds at a time share their operands through its L2.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int rows, int n_tiles, char* lds, Tile& t) {
    int* wave_sum = reinterpret_cast<int*>(lds);       // [8][2]
    Tile* found = reinterpret_cast<Tile*>(lds + 256);
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_in_block();
    const int per = (E + kThreads - 1) / kThreads;
    const int e0 = min(E, tid * per), e1 = min(E, e0 + per);
    int full = 0, tail = 0;
    for (int e = e0; e < e1; ++e) {
        const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], lo), rows);
        full += (hi - lo) / kFullRows;
        tail += (hi - lo) % kFullRows != 0;
    }
    int sf = full, st = tail;
    for (int d = 1; d < kWave; d <<= 1) {
        const int a = __shfl_up(sf, d), b = __shfl_up(st, d);
        if (lane >= d) sf += a, st += b;
    }
    if (lane == kWave - 1) wave_sum[wave * 2] = sf, wave_sum[wave * 2 + 1] = st;
    if (tid == 0) found->expert = -1;
    __syncthreads();
    int total_f = 0, total_t = 0, before_f = 0, before_t = 0;
    for (int w = 0; w < kThreads / kWave; ++w) {
        if (w == wave) before_f = total_f, before_t = total_t;
        total_f += wave_sum[w * 2], total_t += wave_sum[w * 2 + 1];
    }
    // Exclusive prefix of this thread's experts.
    int pf = before_f + sf - full, pt = before_t + st - tail;
    const int per_f = (total_f * n_tiles + 7) / 8, per_t = (total_t * n_tiles + 7) / 8;
    const int xcd = blockIdx.x % 8, seq = blockIdx.x / 8;
    const bool is_tail = seq >= per_f;
    const int item = is_tail ? xcd * per_t + seq - per_f : xcd * per_f + seq;
    const bool none = is_tail ? (seq - per_f >= per_t || item >= total_t * n_tiles) : item >= total_f * n_tiles;
    if (none) return false;
    for (int e = e0; e < e1; ++e) {
        const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], lo), rows);
        const int m = hi - lo, nf = m / kFullRows, nt = m % kFullRows != 0;
        if (!is_tail && item >= pf * n_tiles && item < (pf + nf) * n_tiles) {
            // Groups of up to 8 row tiles, the column tiles of a group one after
            // the other: the 32 tiles that an XCD works on at a time are then
            // about 8 x 4 and share their operands, also in an expert of many rows.
            const int local = item - pf * n_tiles;
            const int group = local / (8 * n_tiles), in = local % (8 * n_tiles), high = min(8, nf - group * 8);
            *found = {e, lo + (group * 8 + in % high) * kFullRows, kFullRows, in / high, kFullRows};
        }
        if (is_tail && nt && item >= pt * n_tiles && item < (pt + 1) * n_tiles) {
            const int r = m % kFullRows;
            *found = {e, hi - r, r, item - pt * n_tiles, r > 128 ? 256 : r > 64 ? 128 : 64};
        }
        pf += nf, pt += nt;
    }
    __syncthreads();
    t = *found;
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    t.n = __builtin_amdgcn_readfirstlane(t.n);
    t.shape = __builtin_amdgcn_readfirstlane(t.shape);
    __syncthreads();
    return t.expert >= 0;
}

// Workgroups that cover every tile of `rows` rows over E experts.
int64_t tile_grid(int64_t rows, int E, int64_t n_tiles) {
    const int64_t full = rows / kFullRows * n_tiles, tails = std::min<int64_t>(E, rows) * n_tiles;
    return (full + 7) / 8 * 8 + (tails + 7) / 8 * 8;
}

struct MatmulArgs {
    const int32_t* offsets;
    const uint16_t* x;
    const uint16_t* w;
    uint16_t* y;
    int E, rows, k_dim, n_dim;
    uint32_t* err;
};

__device__ __forceinline__ void check_rows(const int32_t* offsets, int E, int rows, uint32_t* err) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && offsets[E] > rows) report(err, EP_DEVERR_CAPACITY);
}

// Waves: WM over rows, 8 / WM over columns; a wave's block is MS x NS sub-tiles
// of 16 x 16.
template <int WM, int MS, bool KN>
__device__ __forceinline__ void matmul_tile(const MatmulArgs& a, const Tile& t, char* lds) {
    constexpr int WN = 8 / WM, NS = 16 / WN, ROWS = WM * MS * 16;
    const int wave = uniform_wave(), wm = wave / WN, wn = wave % WN;
    const int64_t K = a.k_dim, N = a.n_dim;
    const int n0 = t.n * kTileN;
    RowsLoader<ROWS> la;
    const uint32_t x_ld = (uint32_t)K * 2;
    la.init(a.x + (int64_t)t.row0 * K, (uint32_t)t.rows * x_ld,
            [&](int r) { return r < t.rows ? r * x_ld : kBufOutside; });
    RowsReader ra;
    ra.init(wm * MS);
    f32x4 acc[MS][NS] = {};
    const uint16_t* w = a.w + (int64_t)t.expert * N * K;
    if constexpr (KN) {
        ColsLoader lb;
        lb.init(w, N, n0);
        ColsReader<NS> rb;
        rb.init(wn * NS);
        multiply<MS, NS>(la, lb, ra, rb, a.k_dim, lds, acc);
    } else {
        RowsLoader<kTileN> lb;
        const int cols = min((int)N - n0, kTileN);
        lb.init(w + (int64_t)n0 * K, (uint32_t)cols * x_ld,
                [&](int r) { return r < cols ? r * x_ld : kBufOutside; });
        RowsReader rb;
        rb.init(wn * NS);
        multiply<MS, NS>(la, lb, ra, rb, a.k_dim, lds, acc);
    }
    const int i = lane_id() & 15, q = lane_id() >> 4;
#pragma unroll
    for (int mi = 0; mi < MS; ++mi) {
        const int m = (wm * MS + mi) * 16 + i;
        if (m >= t.rows) continue;
        uint16_t* row = a.y + (int64_t)(t.row0 + m) * N;
#pragma unroll
        for (int ni = 0; ni < NS; ++ni) {
            const int n = n0 + (wn * NS + ni) * 16 + q * 4;
            const f32x4 v = acc[mi][ni];
            const u32x2 o = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            if (n < N) *reinterpret_cast<u32x2*>(row + n) = o;
        }
    }
}

template <bool KN>
__global__ __launch_bounds__(kThreads, 2) void matmul_kernel(MatmulArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
    check_rows(a.offsets, a.E, a.rows, a.err);
    Tile t;
    if (!find_tile(a.offsets, a.E, a.rows, (a.n_dim + kTileN - 1) / kTileN, lds, t)) return;
    if (t.shape == 256)
        matmul_tile<2, 8, KN>(a, t, lds);
    else if (t.shape == 128)
        matmul_tile<2, 4, KN>(a, t, lds);
    else
        matmul_tile<1, 4, KN>(a, t, lds);
}

// ---- Gate/up product with SwiGLU and the 8-bit checkpoint -------------------

struct SwigluArgs {
    const int32_t* offsets;
    const uint16_t* x;
    const uint16_t* w13;
    uint16_t* act;
    uint8_t* gu;
    float* scales;
    int E, rows, H, F;
    uint32_t* err;
};

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

// Scale of a block of 128 values with the largest magnitude amax: amax / 448,
// so that the largest value is e4m3's largest; 1 where amax / 448 would be
// too small to invert (all values then round to 0).
__device__ __forceinline__ float block_scale(float amax) { return amax < 1e-33f ? 1.0f : amax / 448.0f; }

// A column tile is 128 values of f: wave wn's columns are gate values of NS / 2
// sub-tiles, then the up values of the same f, so one lane holds both.
template <int WM, int MS, bool SAVE>
__device__ __forceinline__ void swiglu_tile(const SwigluArgs& a, const Tile& t, char* lds) {
    constexpr int WN = 8 / WM, NS = 16 / WN, HS = NS / 2, ROWS = WM * MS * 16;
    const int wave = uniform_wave(), wm = wave / WN, wn = wave % WN;
    const int f0 = t.n * (kTileN / 2);
    RowsLoader<ROWS> la;
    RowsLoader<kTileN> lb;
    const uint32_t ld = (uint32_t)a.H * 2;
    la.init(a.x + (int64_t)t.row0 * a.H, (uint32_t)t.rows * ld, [&](int r) { return r < t.rows ? r * ld : kBufOutside; });
    lb.init(a.w13 + (int64_t)t.expert * 2 * a.F * a.H, (uint32_t)(2 * a.F) * ld, [&](int r) {
        const int in = r % (NS * 16), f = f0 + r / (NS * 16) * (HS * 16) + in % (HS * 16);
        return f < a.F ? (uint32_t)(f + (in < HS * 16 ? 0 : a.F)) * ld : kBufOutside;
    });
    RowsReader ra, rb;
    ra.init(wm * MS);
    rb.init(wn * NS);
    f32x4 acc[MS][NS] = {};
    multiply<MS, NS>(la, lb, ra, rb, a.H, lds, acc);

    const int i = lane_id() & 15, q = lane_id() >> 4;
    const int fw = f0 + wn * HS * 16 + q * 4;
    float* amax = reinterpret_cast<float*>(lds);  // [WN][ROWS][2]
    if constexpr (SAVE) {
#pragma unroll
        for (int mi = 0; mi < MS; ++mi) {
            float g = 0.f, u = 0.f;
#pragma unroll
            for (int ni = 0; ni < HS; ++ni)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    g = fmaxf(g, fabsf(acc[mi][ni][j]));
                    u = fmaxf(u, fabsf(acc[mi][ni + HS][j]));
                }
            g = fmaxf(g, __shfl_xor(g, 16)), u = fmaxf(u, __shfl_xor(u, 16));
            g = fmaxf(g, __shfl_xor(g, 32)), u = fmaxf(u, __shfl_xor(u, 32));
            if (q == 0) {
                float* p = amax + (wn * ROWS + (wm * MS + mi) * 16 + i) * 2;
                p[0] = g, p[1] = u;
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int mi = 0; mi < MS; ++mi) {
        const int m = (wm * MS + mi) * 16 + i;
        if (m >= t.rows) continue;
        const int64_t row = t.row0 + m;
        float gi = 0.f, ui = 0.f;
        if constexpr (SAVE) {
            float g = 0.f, u = 0.f;
#pragma unroll
            for (int w = 0; w < WN; ++w) {
                g = fmaxf(g, amax[(w * ROWS + m) * 2]);
                u = fmaxf(u, amax[(w * ROWS + m) * 2 + 1]);
            }
            g = block_scale(g), u = block_scale(u);
            if (wn == 0 && q == 0) {
                float* s = a.scales + row * (2 * a.F / 128);
                s[t.n] = g, s[a.F / 128 + t.n] = u;
            }
            gi = 1.0f / g, ui = 1.0f / u;
        }
#pragma unroll
        for (int ni = 0; ni < HS; ++ni) {
            const int f = fw + ni * 16;
            if (f >= a.F) continue;
            const f32x4 g = acc[mi][ni], u = acc[mi][ni + HS];
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = g[j] * sigmoid(g[j]) * u[j];
            const u32x2 o = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            *reinterpret_cast<u32x2*>(a.act + row * a.F + f) = o;
            if constexpr (SAVE) {
                uint8_t* c = a.gu + row * 2 * a.F + f;
                *reinterpret_cast<uint32_t*>(c) = pack_e4m3(g[0] * gi, g[1] * gi, g[2] * gi, g[3] * gi);
                *reinterpret_cast<uint32_t*>(c + a.F) = pack_e4m3(u[0] * ui, u[1] * ui, u[2] * ui, u[3] * ui);
            }
        }
    }
}

template <bool SAVE>
__global__ __launch_bounds__(kThreads, 2) void swiglu_kernel(SwigluArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
    check_rows(a.offsets, a.E, a.rows, a.err);
    Tile t;
    if (!find_tile(a.offsets, a.E, a.rows, (a.F + kTileN / 2 - 1) / (kTileN / 2), lds, t)) return;
    if (t.shape == 256)
        swiglu_tile<2, 8, SAVE>(a, t, lds);
    else if (t.shape == 128)
        swiglu_tile<2, 4, SAVE>(a, t, lds);
    else
        swiglu_tile<1, 4, SAVE>(a, t, lds);
}

// ---- Weight gradient ----------------------------------------------------------

struct WgradArgs {
    const int32_t* offsets;
    const uint16_t* dy;
    const uint16_t* x;
    const uint8_t* x8;
    const float* x_scales;
    void* dw;
    int E, rows, n_dim, k_dim;
    uint32_t* err;
};

// The FP8 rows of a step: each thread fetches 32 values (two 16-byte vectors) of
// one memory row with their block's scale into registers, and half a step
// later writes them to LDS as bf16 in the columns layout. The value is rounded
// to bf16 once (2^-8 of it, against e4m3's own 2^-4) because the matrix
// instruction multiplies bf16.
struct Fp8Loader {
    static constexpr int kLoads = 0;  // copies to LDS
    const uint8_t* p;
    const float* s;
    int64_t ld;
    int row, col;
    bool in_cols;
    u32x4 v[2];
    float scale;

    __device__ __forceinline__ void init(const uint8_t* x8, const float* scales, int64_t k_dim, int col0) {
        row = threadIdx.x >> 3;
        col = (threadIdx.x & 7) * 32;
        ld = k_dim;
        in_cols = col0 + col < k_dim;
        p = x8 + row * ld + col0 + col;
        s = scales + row * (ld / 128) + (col0 + col) / 128;
    }
    __device__ __forceinline__ void copy(int, uint32_t) {}
    __device__ __forceinline__ void begin(int k0, int k_dim) {
        const u32x4 zero = {0u, 0u, 0u, 0u};
        v[0] = v[1] = zero;
        scale = 0.f;
        if (k0 + row < k_dim && in_cols) {
            v[0] = ld16(p + k0 * ld);
            v[1] = ld16(p + k0 * ld + 16);
            scale = s[k0 * (ld / 128)];
        }
    }
    __device__ __forceinline__ void stage(char* lds) const {
        const int f = (row & 3) | (((row >> 3) & 3) << 2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t o[8];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[h][w], false);
                const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[h][w], true);
                o[2 * w] = pack_bf16(lo[0] * scale, lo[1] * scale);
                o[2 * w + 1] = pack_bf16(hi[0] * scale, hi[1] * scale);
            }
            char* d = lds + row * 512 + (((col / 16 + h) ^ f) << 5);
            *reinterpret_cast<u32x4*>(d) = {o[0], o[1], o[2], o[3]};
            *reinterpret_cast<u32x4*>(d + 16) = {o[4], o[5], o[6], o[7]};
        }
    }
};

template <bool FP8, bool F32>
__global__ __launch_bounds__(kThreads, 2) void wgrad_kernel(WgradArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
    constexpr int WN = 4, MS = 8, NS = 4;
    check_rows(a.offsets, a.E, a.rows, a.err);
    const int tiles_k = (a.k_dim + kTileN - 1) / kTileN, tiles_n = (a.n_dim + kFullRows - 1) / kFullRows;
    const int total = a.E * tiles_k * tiles_n, per = (total + 7) / 8;
    const int item = (blockIdx.x % 8) * per + blockIdx.x / 8;
    if ((int)blockIdx.x / 8 >= per || item >= total) return;
    const int e = item / (tiles_k * tiles_n), local = item % (tiles_k * tiles_n);
    const int n0 = local % tiles_n * kFullRows, k0 = local / tiles_n * kTileN;
    const int lo = min(max(a.offsets[e], 0), a.rows), hi = min(max(a.offsets[e + 1], lo), a.rows);
    const int rows = __builtin_amdgcn_readfirstlane(hi - lo);
    const int row0 = __builtin_amdgcn_readfirstlane(lo);

    const int wave = uniform_wave(), wm = wave / WN, wn = wave % WN;
    f32x4 acc[MS][NS] = {};
    ColsLoader la;
    la.init(a.dy + (int64_t)row0 * a.n_dim, a.n_dim, n0);
    ColsReader<MS> ra;
    ra.init(wm * MS);
    ColsReader<NS> rb;
    rb.init(wn * NS);
    if constexpr (!FP8) {
        ColsLoader lb;
        lb.init(a.x + (int64_t)row0 * a.k_dim, a.k_dim, k0);
        multiply<MS, NS>(la, lb, ra, rb, rows, lds, acc);
    } else {
        Fp8Loader lb;
        lb.init(a.x8 + (int64_t)row0 * a.k_dim, a.x_scales + (int64_t)row0 * (a.k_dim / 128), a.k_dim, k0);
        multiply<MS, NS>(la, lb, ra, rb, rows, lds, acc);
    }
    const int i = lane_id() & 15, q = lane_id() >> 4;
#pragma unroll
    for (int mi = 0; mi < MS; ++mi) {
        const int n = n0 + (wm * MS + mi) * 16 + i;
        if (n >= a.n_dim) continue;
        const int64_t row = ((int64_t)e * a.n_dim + n) * a.k_dim;
#pragma unroll
        for (int ni = 0; ni < NS; ++ni) {
            const int k = k0 + (wn * NS + ni) * 16 + q * 4;
            if (k >= a.k_dim) continue;
            const f32x4 v = acc[mi][ni];
            if constexpr (F32) {
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.dw) + row + k) = v;
            } else {
                const u32x2 o = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dw) + row + k) = o;
            }
        }
    }
}

template <class Args>
hipError_t launch_tiles(void (*kernel)(Args), int64_t grid, const Args& a, hipStream_t st) {
    if (grid <= 0) return hipSuccess;
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

uint32_t* err_words(char* ws) { return reinterpret_cast<uint32_t*>(ws); }

}  // namespace

int64_t expert_matmul_grid(int64_t rows, int E, int n_dim) {
    return tile_grid(rows, E, (n_dim + kTileN - 1) / kTileN);
}
int64_t expert_swiglu_grid(int64_t rows, int E, int F) {
    return tile_grid(rows, E, (F + kTileN / 2 - 1) / (kTileN / 2));
}
int64_t expert_wgrad_grid(int E, int n_dim, int k_dim) {
    const int64_t total = (int64_t)E * ((n_dim + kFullRows - 1) / kFullRows) * ((k_dim + kTileN - 1) / kTileN);
    return (total + 7) / 8 * 8;
}

hipError_t launch_expert_matmul(const ep_shape& s, const ep_layout& L, const uint16_t* x, int64_t rows, int k_dim,
                                const uint16_t* w, int n_dim, int order, uint16_t* y, char* ws, hipStream_t st) {
    const MatmulArgs a = {L.expert_offsets, x, w, y, s.E, (int)rows, k_dim, n_dim, err_words(ws)};
    return launch_tiles(order == EP_WEIGHT_KN ? matmul_kernel<true> : matmul_kernel<false>,
                        expert_matmul_grid(rows, s.E, n_dim), a, st);
}

hipError_t launch_expert_swiglu(const ep_shape& s, const ep_layout& L, const uint16_t* x, int64_t rows,
                                const uint16_t* w13, int F, uint16_t* act, uint8_t* gu, float* scales, char* ws,
                                hipStream_t st) {
    const SwigluArgs a = {L.expert_offsets, x, w13, act, gu, scales, s.E, (int)rows, s.H, F, err_words(ws)};
    return launch_tiles(gu ? swiglu_kernel<true> : swiglu_kernel<false>, expert_swiglu_grid(rows, s.E, F), a, st);
}

hipError_t launch_expert_wgrad(const ep_shape& s, const ep_layout& L, const uint16_t* dy, int64_t rows, int n_dim,
                               const uint16_t* x, const uint8_t* x8, const float* x_scales, int k_dim, void* dw,
                               int dtype, char* ws, hipStream_t st) {
    const WgradArgs a = {L.expert_offsets, dy, x, x8, x_scales, dw, s.E, (int)rows, n_dim, k_dim, err_words(ws)};
    void (*const kernels[2][2])(WgradArgs) = {{wgrad_kernel<false, false>, wgrad_kernel<false, true>},
                                              {wgrad_kernel<true, false>, wgrad_kernel<true, true>}};
    return launch_tiles(kernels[x8 != nullptr][dtype == EP_GRAD_F32], expert_wgrad_grid(s.E, n_dim, k_dim), a, st);
}

}  // namespace ep
