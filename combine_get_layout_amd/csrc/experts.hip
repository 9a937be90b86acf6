// experts.hip -- products of the expert-grouped rows with the experts' weights
// on gfx950: ep_expert_matmul, ep_expert_swiglu and ep_expert_wgrad.
//
// Rows i of expert e are [expert_offsets[e], expert_offsets[e+1]).
//   matmul  y[i][n]  = sum_k x[i][k] W[e][n][k]   (or W[e][k][n])
//   swiglu  g = x W13[e][0:F]^T, u = x W13[e][F:2F]^T, act = silu(g) u
//   wgrad   dW[e][n][k] = sum_{i of e} dy[i][n] x[i][k]
#include <algorithm>
#include <type_traits>

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
// "Rows" layout: rows of 64 contracted values (128 bytes, eight 16-byte
// chunks). Chunk c of row r lies at chunk c ^ f(r). A wave's 16-byte reads go
// through the banks (64 x 4 bytes) in groups of 16 lanes such as {0-3, 12-15,
// 20-27}; f(r) = (r >> 1) & 7 serves lanes that read 16 rows in a run,
// pairs_swizzle those that read rows 8 a + b (a, b = 0..3), both without
// conflicts.
//
// "Columns" layout: 64 contracted rows of 256 values (512 bytes, sixteen
// 32-byte blocks). Block b of row k lies at block b ^ cols_swizzle(k): the 16
// rows that a wave's transposing read touches then cover the banks evenly.
//
// Steps of 64 rather than 32 indices, so that every copy takes whole 128-byte
// lines: with 64-byte pieces the copies filled the L2's requests (6% less at 32
// experts of 1,024 x 7168 x 4096, else alike).
__device__ __forceinline__ int pairs_swizzle(int r) { return ((r >> 1) & 1) | ((r >> 3) & 3) << 1; }
__device__ __forceinline__ int cols_swizzle(int k) { return (k & 3) | ((k >> 3) & 3) << 2; }

// The loaders keep their place in scalar registers; a lane's offsets depend on
// the launch alone, so turning to another tile costs no vector register.

// A tile operand whose contracted index is contiguous in memory: 256 rows,
// first (PAIRS false) or second operand.
template <bool PAIRS>
struct RowsLoader {
    static constexpr int kLoads = 4;         // copies of a step, 64 rows each
    static constexpr int kYounger = kLoads;  // loads of later steps at the wait for a step
    static constexpr bool kStaged = false;   // copies go to LDS as they are
    uint32_t off[kLoads];  // of this lane's 16 bytes in each copy
    int k;                 // their first contracted index within a step
    uint32_t lds_wave;     // LDS bytes before this wave's part of a copy
    const char* p;
    uint32_t bytes;  // of the tile's rows that exist; the rest read as zero
    int k_dim;       // contracted indices; 0: every step is past the end
    u32x4 d;         // the step under way
    uint32_t far;

    // row: memory row of LDS row r < 256 of the tile.
    template <class Row>
    __device__ __forceinline__ void init(uint32_t ld_bytes, Row row) {
        const int lane = lane_id(), r = wave_in_block() * 8 + (lane >> 3);
        const int chunk = (lane & 7) ^ (PAIRS ? pairs_swizzle(r) : (r >> 1) & 7);
        k = chunk * 8;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) off[j] = row(j * 64 + r) * ld_bytes + chunk * 16;
        lds_wave = uniform_wave() * 8 * 128;
    }
    __device__ __forceinline__ void start(const void* base, uint32_t n_bytes, int contracted) {
        p = static_cast<const char*>(base);
        bytes = n_bytes;
        k_dim = contracted;
    }
    // Turns to the step whose first index is k0 (zeros past k_dim).
    __device__ __forceinline__ void begin(int k0) {
        d = buf_desc(p + (int64_t)k0 * 2, k0 < k_dim ? bytes - (uint32_t)k0 * 2 : 0u);
        far = k0 + k < k_dim ? 0u : kBufFar;
    }
    // Requests part j of kLoads of that step into LDS.
    __device__ __forceinline__ void copy(int j, uint32_t lds) {
        copy16_to_lds(d, off[j] + far, lds + lds_wave + j * 8192);
    }
    __device__ __forceinline__ void stage(int, char*) {}
    __device__ __forceinline__ void fetch(int) {}
};

// A tile operand whose 256 columns are contiguous in memory (one contracted
// index per memory row of ld values).
struct ColsLoader {
    static constexpr int kLoads = 4;  // copies of a step, 16 contracted rows each
    static constexpr int kYounger = kLoads;
    static constexpr bool kStaged = false;
    uint32_t off[kLoads];
    uint32_t lds_wave;
    int64_t ld_bytes;
    const char* p;
    uint32_t col_bytes;  // bytes of a row before the tile's first column
    int k_dim;
    u32x4 d;

    __device__ __forceinline__ void init(int64_t ld) {
        ld_bytes = ld * 2;
        const int lane = lane_id();
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int r = j * 16 + wave_in_block() * 2 + (lane >> 5);
            const int block = ((lane & 31) >> 1) ^ cols_swizzle(r);
            off[j] = (uint32_t)(r * ld_bytes) + block * 32 + (lane & 1) * 16;
        }
        lds_wave = uniform_wave() * 2 * 512;
    }
    __device__ __forceinline__ void start(const void* base, int contracted, int col0) {
        p = static_cast<const char*>(base) + (int64_t)col0 * 2;
        col_bytes = col0 * 2;
        k_dim = contracted;
    }
    __device__ __forceinline__ void begin(int k0) {
        const int rows = min(k_dim - k0, kStep);
        d = buf_desc(p + (int64_t)k0 * ld_bytes, rows > 0 ? (uint32_t)(rows * (int)ld_bytes) - col_bytes : 0u);
    }
    __device__ __forceinline__ void copy(int j, uint32_t lds) { copy16_to_lds(d, off[j], lds + lds_wave + j * 8192); }
    __device__ __forceinline__ void stage(int, char*) {}
    __device__ __forceinline__ void fetch(int) {}
};

// The FP8 rows of a step as second operand: each thread fetches 32 values (two
// 16-byte vectors) of one memory row with their block's scale into registers,
// and a step later writes them to LDS as bf16 in the columns layout, a quarter
// at a time between the matrix instructions. The value is rounded to bf16
// once (2^-8 of it, against e4m3's own 2^-4) because the matrix instruction
// multiplies bf16.
struct Fp8Loader {
    static constexpr int kLoads = 0;    // copies to LDS
    static constexpr int kYounger = 3;  // the next step's fetch
    static constexpr bool kStaged = true;
    const uint8_t* p;
    const float* s;
    int64_t ld;
    int row0, k_dim, col0;
    bool outside;
    u32x4 v[2];
    float scale;

    __device__ __forceinline__ void init(const uint8_t* x8, const float* scales, int64_t ld_) {
        p = x8, s = scales, ld = ld_;
    }
    __device__ __forceinline__ void start(int first, int contracted, int col) { row0 = first, k_dim = contracted, col0 = col; }
    __device__ __forceinline__ void copy(int, uint32_t) {}
    __device__ __forceinline__ void begin(int) {}
    // Always three loads (wait counts rely on it); outside the expert's rows and
    // the columns they read the array's first values and count as zero.
    __device__ __forceinline__ void fetch(int k0) {
        const int row = k0 + (threadIdx.x >> 3), col = col0 + (threadIdx.x & 7) * 32;
        const bool in = row < k_dim && col < ld;
        const int64_t r = in ? row0 + row : 0;
        const int c = in ? col : 0;
        v[0] = ld16(p + r * ld + c);
        v[1] = ld16(p + r * ld + c + 16);
        scale = s[r * (ld / 128) + c / 128];
        outside = !in;
    }
    __device__ __forceinline__ void stage(int part, char* lds) const {
        const int row = threadIdx.x >> 3, block = (threadIdx.x & 7) * 2 + (part >> 1);
        uint32_t o[4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int q = outside ? 0 : (int)v[part >> 1][(part & 1) * 2 + w];
            const float f = outside ? 0.f : scale;
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(q, false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(q, true);
            o[2 * w] = pack_bf16(lo[0] * f, lo[1] * f);
            o[2 * w + 1] = pack_bf16(hi[0] * f, hi[1] * f);
        }
        char* d = lds + row * 512 + ((block ^ cols_swizzle(row)) << 5) + (part & 1) * 16;
        *reinterpret_cast<u32x4*>(d) = {o[0], o[1], o[2], o[3]};
    }
};

// 16 x 32 fragments of the step at lds: sub-tile s, half `half` of the
// contracted indices. First operand: sub-tile s is rows (or columns) 16 s .. +
// 15. Second operand ("pairs"): sub-tiles 2 p + u, u = 0, 1, share 32 columns,
// u holding columns 8 a + 4 u + b (a, b = 0..3) as its 16, so that a lane's
// results of both are 8 consecutive columns: 16-byte stores of bf16.
struct RowsReader {
    uint32_t base[2];
    __device__ __forceinline__ void init(int first_row) {
        const int i = lane_id() & 15, q = lane_id() >> 4;
        const uint32_t row = (first_row + i) * 128;
        base[0] = row + ((q ^ (i >> 1)) * 16);
        base[1] = row + (((q + 4) ^ (i >> 1)) * 16);
    }
    __device__ __forceinline__ bf16x8 read(const char* lds, int s, int half) const {
        return *reinterpret_cast<const bf16x8*>(lds + base[half] + s * 2048);
    }
};
// STEP: LDS rows from one sub-tile of a pair to the other.
template <int STEP>
struct RowsPairReader {
    uint32_t base[2];
    __device__ __forceinline__ void init(int first_col) {
        const int i = lane_id() & 15, q = lane_id() >> 4;
        const int r = (i >> 2) * 8 + (i & 3);
        const uint32_t row = (first_col + r) * 128;
        base[0] = row + ((q ^ pairs_swizzle(r)) * 16);
        base[1] = row + (((q + 4) ^ pairs_swizzle(r)) * 16);
    }
    __device__ __forceinline__ bf16x8 read(const char* lds, int s, int half) const {
        return *reinterpret_cast<const bf16x8*>(lds + base[half] + (s >> 1) * 4096 + (s & 1) * STEP * 128);
    }
};
// The columns layout is read by the transposing instruction: each 16-lane
// group reads 4 contracted rows of 4 pieces of 4 values and receives them
// transposed: lane i gets the 4 rows' values of column i % 4 of piece i / 4.
template <bool PAIRS>
struct ColsReader {
    uint32_t base;
    __device__ __forceinline__ void init(int first_col) {  // a multiple of 128, with PAIRS of 32
        const int i = lane_id() & 15, q = lane_id() >> 4, piece = i & 3;
        const int k = q * 8 + (i >> 2), b0 = first_col / 16;
        base = PAIRS ? k * 512 + (((b0 + (piece >> 1)) ^ cols_swizzle(k)) << 5) + (piece & 1) * 16
                     : k * 512 + ((b0 ^ cols_swizzle(k)) << 5) + piece * 8;
    }
    // Sub-tiles (PAIRS: pairs of them) differ in address bits that are clear in
    // b0, so that the swizzled address is reached by an exclusive or.
    __device__ __forceinline__ bf16x8 read(const char* lds, int s, int half) const {
        const char* p = lds + ((PAIRS ? base ^ ((s >> 1) << 6) : base ^ (s << 5)) + (PAIRS ? (s & 1) * 8 : 0) + half * 16384);
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
// read from (a_lds, b_lds, half), in MS groups of NS matrix instructions, each
// behind its share of the reads and of the copies: copies issued in one go
// would stand in the waves' way until the memory pipeline has taken them all
// (16 clocks each).
template <int MS, int NS, class RA, class RB, class Copies>
__device__ __forceinline__ void half_step(const RA& ra, const RB& rb, const char* a_lds, const char* b_lds, int half,
                                          const Fragments<MS, NS>& cur, Fragments<MS, NS>& next,
                                          f32x4 (&acc)[MS][NS], Copies copies) {
    constexpr int R = MS + NS;
#pragma unroll
    for (int g = 0; g < MS; ++g) {
#pragma unroll
        for (int r = g * R / MS; r < (g + 1) * R / MS; ++r) {
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

// The slots of the steps s and s + 1 and (second operand) the free one.
struct Ring {
    int a_now, a_next, b_now, b_next, b_free;
};
__device__ __forceinline__ Ring first_ring() { return {0, kPart, kRingB, kRingB + kPart, kRingB + 2 * kPart}; }

// Requests the first two steps of a tile (three of FP8 rows, which it converts).
template <class LA, class LB>
__device__ __forceinline__ void first_steps(LA& la, LB& lb, char* lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_address(lds));
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        la.begin(s * kStep);
        lb.begin(s * kStep);
        lb.fetch(s * kStep);
#pragma unroll
        for (int c = 0; c < LA::kLoads; ++c) la.copy(c, at + s * kPart);
#pragma unroll
        for (int c = 0; c < LB::kLoads; ++c) lb.copy(c, at + kRingB + s * kPart);
#pragma unroll
        for (int c = 0; c < 4; ++c) lb.stage(c, lds + kRingB + s * kPart);
    }
    lb.fetch(2 * kStep);
}

// One tile's product: acc[mi][ni] += rows sub-tile mi times columns sub-tile
// ni. Each half of a step is multiplied from registers while the fragments of
// the next half are read from LDS, with one barrier per step. All of the LDS
// holds steps: two of the first operand, three of the second. In the first half
// of step s the copies of the second operand's step s + 2 are issued (into the
// slot of step s - 1), in the second half those of the first operand's (into
// the slot of step s, whose last fragments have then been read): one for each
// four matrix instructions from the half's start, so that they have nearly one
// and nearly one and a half step's time to arrive.
//
// Bound: a step of a full tile is 1.08 us of matrix instructions at the 1.9 GHz
// that the card holds under them, and takes 1.5: 1,390 TFLOP/s at 32 experts of
// 1,024 x 7168 x 4096, beside 1,580 of a large library product. What is missing
// are copies that arrive late (all of them from cache: 1,540; neither copies
// nor LDS reads: 1,665). One workgroup per CU: a second would halve the tiles,
// and with them the use that is made of what is read.
//
// Two forms, by what measured better (TFLOP/s at that size, each on the same
// card). `multiply`, a tile of its own: from first_steps, which the caller
// issues beside the results of the tile before, two steps to a turn of the
// loop, so that the slots are constants: products 1,385 (1,349 streamed), with
// KN weights 1,408 (1,363). `multiply_stream`: steps past the tile's last are
// the next tile's first, to which `next` turns the loaders, so that the copies
// have no gap between short tiles; the slots go round in registers: weight
// gradients (16 steps a tile) 1,135 (1,098 by tiles of their own), from FP8
// rows 984 (936).
template <int MS, int NS, class LA, class LB, class RA, class RB>
__device__ __forceinline__ void multiply(LA& la, LB& lb, const RA& ra, const RB& rb, int k_dim, char* lds,
                                         f32x4 (&acc)[MS][NS]) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_address(lds));
    const int steps = (k_dim + kStep - 1) / kStep;
    constexpr int kCopiesA = (MS * NS * 8 + 63) / 64;  // of the tile's MS x 16 x NS / 2 rows, 64 each
    wait_copies<0>();
    barrier_only();
    Fragments<MS, NS> f[2];
    Ring r = first_ring();
#pragma unroll
    for (int i = 0; i < NS; ++i) f[0].b[i] = rb.read(lds + r.b_now, i, 0);
#pragma unroll
    for (int i = 0; i < MS; ++i) f[0].a[i] = ra.read(lds, i, 0);
    for (int s = 0; s < steps; s += 2) {
#pragma unroll
        for (int slot = 0; slot < 2; ++slot) {
            if (slot && s + 1 >= steps) break;
            lb.begin((s + slot + 2) * kStep);
            half_step<MS, NS>(ra, rb, lds + slot * kPart, lds + r.b_now, 1, f[0], f[1], acc, [&](int g) {
                if (g < LB::kLoads) lb.copy(g, at + r.b_free);
            });
            wait_copies<LB::kYounger>();
            barrier_only();
            la.begin((s + slot + 2) * kStep);
            half_step<MS, NS>(ra, rb, lds + (slot ^ 1) * kPart, lds + r.b_next, 0, f[1], f[0], acc, [&](int g) {
                // Copies of rows that the tile's shape does not have are left out.
                if (g < kCopiesA) la.copy(g, at + slot * kPart);
            });
            r = {r.a_next, r.a_now, r.b_next, r.b_free, r.b_now};
        }
    }
    keep(f[0]);
    wait_copies<0>();  // none may land after the slots have been handed on
    settle(acc);
    barrier_only();
}

// Steps of a streamed tile: as many at least as are requested ahead (three of
// FP8 rows), so that these never reach past the next tile.
template <class LB>
__device__ __forceinline__ int stream_steps(int k_dim) {
    return max(LB::kStaged ? 3 : 2, (k_dim + kStep - 1) / kStep);
}

// The streamed form. STORES: at least so many stores of the tile before were
// issued behind its last copies (if `behind`); they need not have finished in
// the first step.
template <int MS, int NS, int STORES, class LA, class LB, class RA, class RB, class Next>
__device__ __forceinline__ void multiply_stream(LA& la, LB& lb, const RA& ra, const RB& rb, int steps, char* lds,
                                                Ring& r, bool behind, f32x4 (&acc)[MS][NS], Next next) {
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_address(lds));
    Fragments<MS, NS> f[2];
#pragma unroll
    for (int i = 0; i < NS; ++i) f[0].b[i] = rb.read(lds + r.b_now, i, 0);
#pragma unroll
    for (int i = 0; i < MS; ++i) f[0].a[i] = ra.read(lds + r.a_now, i, 0);
    auto ahead = [&](int s) { return (s < steps ? s : s - steps) * kStep; };
    if (!LB::kStaged) {
        if (steps == 2) next.b();
        lb.begin(ahead(2));
    }
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
        half_step<MS, NS>(ra, rb, lds + r.a_now, lds + r.b_now, 1, f[0], f[1], acc, [&](int g) {
            if (g < LB::kLoads) lb.copy(g, at + r.b_free);
            if (g == MS - 1) {
                if (s + 2 == steps) next.a();
                la.begin(ahead(s + 2));
            }
        });
        if (behind)
            wait_copies<LB::kYounger + STORES>();
        else
            wait_copies<LB::kYounger>();
        behind = false;
        barrier_only();
        half_step<MS, NS>(ra, rb, lds + r.a_next, lds + r.b_next, 0, f[1], f[0], acc, [&](int g) {
            if (LB::kStaged && g < 4) lb.stage(g, lds + r.b_free);
            if (g < LA::kLoads) la.copy(g, at + r.a_now);
            if (g == (LB::kStaged ? 4 : MS - 1)) {
                if (s + 3 == steps) next.b();
                if (LB::kStaged)
                    lb.fetch(ahead(s + 3));
                else
                    lb.begin(ahead(s + 3));
            }
        });
        r = {r.a_next, r.a_now, r.b_next, r.b_free, r.b_now};
    }
    keep(f[0]);
    settle(acc);
}

// ---- Tiles of ragged experts ------------------------------------------------

struct Tile {
    int expert;
    int row0;  // first row of the tile
    int rows;  // rows of the tile that exist
    int height;  // rows that the tile's shape holds, at most 256
    int n;     // column tile
};

// The tiles of a launch: every expert's m rows are cut evenly into ceil(m / 256)
// row tiles (in multiples of 32 rows), times `n_tiles`. Workgroups go to the 8
// XCDs in turn; each XCD takes a contiguous run of the tiles, and its workgroups
// take them in turn: within an expert groups of up to 8 row tiles, the column
// tiles of a group one after the other, so that the 32 tiles that an XCD works
// on at a time are about 8 x 4 (4 x 8 at 1,024 rows) and, being of one height
// and so in step, share their operands through its L2. Full tiles and a short
// last one lose that: 32 experts of 1,040 rows (gate/up product, 7168 x 2048)
// took 1,846 us with the short tiles beside the full ones, 1,716 with them at
// the end, where they read all the weights again.
struct Tiles {
    const int32_t* offsets;
    int rows, n_tiles;
    int per;  // experts of a lane (each wave covers all and searches for itself)
    int E;
    int before;  // row tiles of the experts before this lane's
    int total;

    // Rows [lo, lo + m) of expert e.
    __device__ __forceinline__ void bounds(int e, int& lo, int& m) const {
        lo = min(max(offsets[e], 0), rows);
        m = min(max(offsets[e + 1], lo), rows) - lo;
    }
    __device__ __forceinline__ static int row_tiles(int m) { return (m + kFullRows - 1) / kFullRows; }

    // Offsets that are negative or decrease give no tiles (of the latter their number
    // might pass 32 bits).
    __device__ __forceinline__ void init(const int32_t* offs, int experts, int n_rows, int n, uint32_t* err) {
        offsets = offs, rows = n_rows, n_tiles = n, E = experts;
        per = (E + kWave - 1) / kWave;
        const int lane = lane_id(), e0 = min(E, lane * per), e1 = min(E, e0 + per);
        int count = 0;
        bool bad = false;
        for (int e = e0; e < e1; ++e) {
            int lo, m;
            bounds(e, lo, m);
            count += row_tiles(m);
            bad |= offsets[e] < 0 || offsets[e + 1] < offsets[e];
        }
        bad = __ballot(bad);
        int sum = count;
        for (int d = 1; d < kWave; d <<= 1) {
            const int v = __shfl_up(sum, d);
            if (lane >= d) sum += v;
        }
        before = sum - count;
        total = bad ? 0 : readlane(sum, kWave - 1) * n_tiles;
        if (blockIdx.x == 0 && threadIdx.x == 0 && (bad || offsets[E] > rows)) report(err, EP_DEVERR_CAPACITY);
    }
    // The seq-th tile of this workgroup's XCD; false if there is none.
    __device__ __forceinline__ bool find(int seq, Tile& t) const {
        const int share = (total + 7) / 8, item = (int)(blockIdx.x % 8) * share + seq;
        if (seq >= share || item >= total) return false;
        const int target = item / n_tiles;  // lies in its expert's range of row tiles
        const int e0 = min(E, lane_id() * per), e1 = min(E, e0 + per);
        int f = before, at = -1, lo0 = 0, m0 = 0, f0 = 0;
        for (int e = e0; e < e1; ++e) {
            int lo, m;
            bounds(e, lo, m);
            const int n = row_tiles(m);
            if (target >= f && target < f + n) at = e, lo0 = lo, m0 = m, f0 = f;
            f += n;
        }
        const int src = __ffsll((unsigned long long)__ballot(at >= 0)) - 1;
        const int m = readlane(m0, src);
        const int local = item - readlane(f0, src) * n_tiles, group = local / (8 * n_tiles);
        const int in = local % (8 * n_tiles), high = min(8, row_tiles(m) - group * 8);
        t.height = ((m + row_tiles(m) - 1) / row_tiles(m) + 31) / 32 * 32;
        const int row = (group * 8 + in % high) * t.height;
        t.expert = readlane(at, src);
        t.row0 = readlane(lo0, src) + row;
        t.rows = min(t.height, m - row);  // at least 1: all tiles but the last hold at most (tiles - 1) * 256 < m
        t.n = in / high;
        return true;
    }
};

// Most tiles of `rows` rows over E experts.
int64_t most_tiles(int64_t rows, int E, int64_t n_tiles) {
    return (rows / kFullRows + std::min<int64_t>(E, rows)) * n_tiles;
}

struct MatmulArgs {
    const int32_t* offsets;
    const uint16_t* x;
    const uint16_t* w;
    uint16_t* y;
    int E, rows, k_dim, n_dim;
    uint32_t* err;
};

// The products' loaders, turned to a tile one operand after the other.
template <bool KN>
struct MatmulLoaders {
    const MatmulArgs& m;
    RowsLoader<false> a;
    std::conditional_t<KN, ColsLoader, RowsLoader<true>> b;

    __device__ __forceinline__ void init() {
        a.init((uint32_t)m.k_dim * 2, [](int r) { return r; });
        if constexpr (KN)
            b.init(m.n_dim);
        else
            b.init((uint32_t)m.k_dim * 2, [](int r) { return r; });
    }
    __device__ __forceinline__ void start_a(const Tile& t) {
        a.start(m.x + (int64_t)t.row0 * m.k_dim, (uint32_t)t.rows * m.k_dim * 2, m.k_dim);
    }
    __device__ __forceinline__ void start_b(const Tile& t) {
        const uint16_t* w = m.w + (int64_t)t.expert * m.n_dim * m.k_dim;
        const int n0 = t.n * kTileN;
        if constexpr (KN)
            b.start(w, m.k_dim, n0);
        else
            b.start(w + (int64_t)n0 * m.k_dim, (uint32_t)min(m.n_dim - n0, kTileN) * m.k_dim * 2, m.k_dim);
    }
};
// Calls f(waves over rows, sub-tiles of a wave along rows) for a tile height.
// The matrix instructions of rows that a tile does not have are spared: 32
// experts of 7168 x 4096 took 312, 335, 355, 374, 401, 860 and 1,582 us with 40,
// 100, 150, 184, 216, 520 and 1,040 rows, and 336, 369, 391, 401, 415, 986 and
// 1,668 us with 256-row tiles alone.
template <int V>
using Int = std::integral_constant<int, V>;
template <class F>
__device__ __forceinline__ void by_height(int height, F f) {
    if (height > 224)
        f(Int<2>(), Int<8>());
    else if (height > 192)
        f(Int<2>(), Int<7>());
    else if (height > 160)
        f(Int<2>(), Int<6>());
    else if (height > 128)
        f(Int<2>(), Int<5>());
    else if (height > 64)
        f(Int<2>(), Int<4>());
    else
        f(Int<1>(), Int<4>());
}

// A wave's block of results, MS x NS sub-tiles at (row0, col0) of a row-major
// matrix of `cols` columns, as bf16 or 32-bit: 8 consecutive columns a lane and
// pair of sub-tiles. The addresses are a scalar base and one offset per lane.
// rows_left, cols_left: of the matrix from (row0, col0) on. STREAM: bf16 results
// go past the caches in whole lines (weight gradients, 1.9 GB beside 2.9 GB of
// reads that L2 serves: 1,143 against 1,120 TFLOP/s; the products' rows, which
// the next call reads, lose 1% by it).
template <bool F32, bool STREAM, int MS, int NS>
__device__ __forceinline__ void store_block(void* out, int64_t row0, int col0, int cols, int rows_left, int cols_left,
                                            const f32x4 (&acc)[MS][NS]) {
    constexpr int kSize = F32 ? 4 : 2;
    const int i = lane_id() & 15, q = lane_id() >> 4;
    char* base = static_cast<char*>(out) + (row0 * cols + col0) * kSize;
    const bool inside = rows_left >= MS * 16 && cols_left >= NS * 16;  // no edge in the block
    if constexpr (STREAM && !F32 && NS == 4) {
        // A lane's two pieces of 16 bytes lie 64 bytes apart. Lanes 0-7 of each 16
        // trade the second against the first of lanes 8-15, eight rows on, so
        // that a store fills whole lines of 128 bytes, of 8 rows.
        const bool upper = i >= 8;
        const int row = i & 7, col = (upper ? 32 : 0) + q * 8;
        const uint32_t lane_off = (uint32_t)(row * cols + col) * kSize;
#pragma unroll
        for (int mi = 0; mi < MS; ++mi) {
            u32x4 p[2], t;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const f32x4 v = acc[mi][2 * u], w = acc[mi][2 * u + 1];
                p[u] = u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3])};
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int give = (int)(upper ? p[0][d] : p[1][d]);
                t[d] = (uint32_t)__builtin_amdgcn_update_dpp(0, give, 0x128, 0xf, 0xf, false);  // row_ror:8
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!inside && (mi * 16 + h * 8 + row >= rows_left || col >= cols_left)) continue;
                char* o = base + (int64_t)(mi * 16 + h * 8) * cols * kSize + lane_off;
                u32x4 b;
#pragma unroll
                for (int d = 0; d < 4; ++d) b[d] = h == 0 ? (upper ? t[d] : p[0][d]) : (upper ? p[1][d] : t[d]);
                st16_stream(o, b);
            }
        }
    } else {
        const uint32_t lane_off = (uint32_t)(i * cols + q * 8) * kSize;
#pragma unroll
        for (int mi = 0; mi < MS; ++mi) {
            char* row = base + (int64_t)mi * 16 * cols * kSize;
#pragma unroll
            for (int p = 0; p < NS / 2; ++p) {
                const f32x4 v = acc[mi][2 * p], w = acc[mi][2 * p + 1];
                if (!inside && (mi * 16 + i >= rows_left || p * 32 + q * 8 >= cols_left)) continue;
                char* o = row + p * 32 * kSize + lane_off;
                if constexpr (F32) {
                    *reinterpret_cast<f32x4*>(o) = v;
                    *reinterpret_cast<f32x4*>(o + 16) = w;
                } else {
                    const u32x4 b = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(w[0], w[1]),
                                     pack_bf16(w[2], w[3])};
                    st16(o, b);
                }
            }
        }
    }
}

// Waves: WM over rows, 8 / WM over columns; a wave's block is MS x NS sub-tiles
// of 16 x 16.
template <int WM, int MS, bool KN, class Next>
__device__ __forceinline__ void matmul_tile(const MatmulArgs& a, const Tile& t, MatmulLoaders<KN>& l, char* lds,
                                            Next next) {
    constexpr int WN = 8 / WM, NS = 16 / WN;
    const int wave = uniform_wave(), wm = wave / WN, wn = wave % WN;
    RowsReader ra;
    ra.init(wm * MS * 16);
    std::conditional_t<KN, ColsReader<true>, RowsPairReader<4>> rb;
    rb.init(wn * NS * 16);
    f32x4 acc[MS][NS] = {};
    multiply<MS, NS>(l.a, l.b, ra, rb, a.k_dim, lds, acc);
    next();
    const int m = wm * MS * 16, n = t.n * kTileN + wn * NS * 16;
    store_block<false, false>(a.y, t.row0 + m, n, a.n_dim, t.rows - m, a.n_dim - n, acc);
}

// One workgroup per CU takes tiles until there are none. The first steps of the
// next tile are requested before the results of this one are stored.
template <bool KN>
__global__ __launch_bounds__(kThreads, 2) void matmul_kernel(MatmulArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
    Tiles tiles;
    tiles.init(a.offsets, a.E, a.rows, (a.n_dim + kTileN - 1) / kTileN, a.err);
    MatmulLoaders<KN> l = {a};
    l.init();
    Tile t;
    int seq = blockIdx.x / 8;
    auto start = [&] {
        if (!tiles.find(seq, t)) return false;
        l.start_a(t);
        l.start_b(t);
        first_steps(l.a, l.b, lds);
        return true;
    };
    bool more = start();
    while (more) {
        const Tile now = t;
        auto next = [&] {
            seq += gridDim.x / 8;
            more = start();
        };
        const auto run = [&](auto wm, auto ms) {
            matmul_tile<wm.value, ms.value, KN>(a, now, l, lds, next);
        };
        by_height(now.height, run);
    }
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

// The reciprocal is the instruction's own, within one unit in the last place of
// 32 bits; the product is rounded to bf16 next.
__device__ __forceinline__ float silu_mul(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Scale of a block of 128 values with the largest magnitude amax: amax / 448,
// so that the largest value is e4m3's largest; 1 where amax / 448 would be
// too small to invert (all values then round to 0). The codes are of v * (1 /
// scale), one 32-bit rounding more than v / scale, which moves about 2 of 10^7
// more values over a boundary of e4m3's rounding; divisions took 1% of the
// kernel's time.
__device__ __forceinline__ float block_scale(float amax) { return amax < 1e-33f ? 1.0f : amax / 448.0f; }

struct SwigluLoaders {
    const SwigluArgs& m;
    RowsLoader<false> a;
    RowsLoader<true> b;

    __device__ __forceinline__ void init() {
        const uint32_t ld = (uint32_t)m.H * 2;
        const int F = m.F;
        a.init(ld, [](int r) { return r; });
        b.init(ld, [=](int r) { return r / 64 * 32 + r % 32 + (r % 64 < 32 ? 0 : F); });
    }
    __device__ __forceinline__ void start_a(const Tile& t) {
        a.start(m.x + (int64_t)t.row0 * m.H, (uint32_t)t.rows * m.H * 2, m.H);
    }
    // Gate rows past F are read as up rows; their results are not stored.
    __device__ __forceinline__ void start_b(const Tile& t) {
        const int f0 = t.n * 128;
        b.start(m.w13 + ((int64_t)t.expert * 2 * m.F + f0) * m.H, (uint32_t)(2 * m.F - f0) * m.H * 2, m.H);
    }
};

// A column tile is 128 values of f: of each 64 LDS rows of the second operand
// the first 32 are gate rows, the last 32 the up rows of the same f, so that
// one lane holds both. V: consecutive values of f that a lane holds.
template <int WM, int MS, bool SAVE, class Next>
__device__ __forceinline__ void swiglu_tile(const SwigluArgs& a, const Tile& t, SwigluLoaders& l, char* lds, Next next) {
    constexpr int WN = 8 / WM, NS = 16 / WN, HS = NS / 2, ROWS = WM * MS * 16, V = 4 * HS;
    const int wave = uniform_wave(), wm = wave / WN, wn = wave % WN;
    const int i = lane_id() & 15, q = lane_id() >> 4;
    RowsReader ra;
    RowsPairReader<NS == 4 ? 4 : 32> rb;
    ra.init(wm * MS * 16);
    int f;
    if constexpr (NS == 4) {
        rb.init(wn * 64);
        f = t.n * 128 + wn * 32 + q * 8;
    } else {  // two waves share 64 LDS rows: u tells them apart, sub-tile 0 is gate, 1 up
        rb.init((wn >> 1) * 64 + (wn & 1) * 4);
        f = t.n * 128 + (wn >> 1) * 32 + q * 8 + (wn & 1) * 4;
    }
    f32x4 acc[MS][NS] = {};
    multiply<MS, NS>(l.a, l.b, ra, rb, a.H, lds, acc);
    next();

    float* amax = reinterpret_cast<float*>(lds + first_ring().b_free);  // [WN][ROWS][2]
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
        barrier_only();
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
        if (f >= a.F) continue;
        uint32_t o[V / 2], cg[HS], cu[HS];
#pragma unroll
        for (int ni = 0; ni < HS; ++ni) {
            const f32x4 g = acc[mi][ni], u = acc[mi][ni + HS];
            o[2 * ni] = pack_bf16(silu_mul(g[0], u[0]), silu_mul(g[1], u[1]));
            o[2 * ni + 1] = pack_bf16(silu_mul(g[2], u[2]), silu_mul(g[3], u[3]));
            if constexpr (SAVE) {
                cg[ni] = pack_e4m3(g[0] * gi, g[1] * gi, g[2] * gi, g[3] * gi);
                cu[ni] = pack_e4m3(u[0] * ui, u[1] * ui, u[2] * ui, u[3] * ui);
            }
        }
        __builtin_memcpy(__builtin_assume_aligned(a.act + row * a.F + f, V * 2), o, V * 2);
        if constexpr (SAVE) {
            uint8_t* c = a.gu + row * 2 * a.F + f;
            __builtin_memcpy(__builtin_assume_aligned(c, V), cg, V);
            __builtin_memcpy(__builtin_assume_aligned(c + a.F, V), cu, V);
        }
    }
}

template <bool SAVE>
__global__ __launch_bounds__(kThreads, 2) void swiglu_kernel(SwigluArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
    Tiles tiles;
    tiles.init(a.offsets, a.E, a.rows, (a.F + 127) / 128, a.err);
    SwigluLoaders l = {a};
    l.init();
    Tile t;
    int seq = blockIdx.x / 8;
    auto start = [&] {
        if (!tiles.find(seq, t)) return false;
        l.start_a(t);
        l.start_b(t);
        first_steps(l.a, l.b, lds);
        return true;
    };
    bool more = start();
    while (more) {
        const Tile now = t;
        auto next = [&] {
            seq += gridDim.x / 8;
            more = start();
        };
        const auto run = [&](auto wm, auto ms) {
            swiglu_tile<wm.value, ms.value, SAVE>(a, now, l, lds, next);
        };
        by_height(now.height, run);
    }
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

// Turns the loaders to the tile after (no more steps if there is none).
template <class Loaders, class T>
struct NextTile {
    Loaders& l;
    const T& t;
    bool more;
    __device__ __forceinline__ void a() {
        if (more)
            l.start_a(t);
        else
            l.a.k_dim = 0;
    }
    __device__ __forceinline__ void b() {
        if (more)
            l.start_b(t);
        else
            l.b.k_dim = 0;
    }
};

struct Place {
    int e, n0, k0, row0, rows;
};
template <bool FP8>
struct WgradLoaders {
    const WgradArgs& m;
    ColsLoader a;
    std::conditional_t<FP8, Fp8Loader, ColsLoader> b;

    __device__ __forceinline__ void init() {
        a.init(m.n_dim);
        if constexpr (FP8)
            b.init(m.x8, m.x_scales, m.k_dim);
        else
            b.init(m.k_dim);
    }
    __device__ __forceinline__ void start_a(const Place& t) {
        a.start(m.dy + (int64_t)t.row0 * m.n_dim, t.rows, t.n0);
    }
    __device__ __forceinline__ void start_b(const Place& t) {
        if constexpr (FP8)
            b.start(t.row0, t.rows, t.k0);
        else
            b.start(m.x + (int64_t)t.row0 * m.k_dim, t.rows, t.k0);
    }
};

// Tiles of 256 x 256 of each expert's matrix, all of an expert after the
// other, contracted over the expert's rows; the workgroups of an XCD take a
// contiguous run of them, in groups of up to 8 tiles along n.
template <bool FP8, bool F32>
__global__ __launch_bounds__(kThreads, 2) void wgrad_kernel(WgradArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes];
    constexpr int WN = 4, MS = 8, NS = 4;
    const int tiles_k = (a.k_dim + kTileN - 1) / kTileN, tiles_n = (a.n_dim + kFullRows - 1) / kFullRows;
    const int total = a.E * tiles_k * tiles_n, per = (total + 7) / 8;
    const int first = (blockIdx.x % 8) * per, mine = min(max(total - first, 0), per);
    const int wave = uniform_wave(), wm = wave / WN, wn = wave % WN;
    ColsReader<false> ra;
    ra.init(wm * MS * 16);
    ColsReader<true> rb;
    rb.init(wn * NS * 16);
    WgradLoaders<FP8> l = {a};
    auto place = [&](int seq, Place& t) {
        if (seq >= mine) return false;
        const int item = first + seq;
        t.e = item / (tiles_k * tiles_n);
        const int local = item % (tiles_k * tiles_n);
        const int group = local / (8 * tiles_k), in = local % (8 * tiles_k), high = min(8, tiles_n - group * 8);
        t.n0 = (group * 8 + in % high) * kFullRows;
        t.k0 = in / high * kTileN;
        const int lo = min(max(a.offsets[t.e], 0), a.rows), hi = min(max(a.offsets[t.e + 1], lo), a.rows);
        t.row0 = __builtin_amdgcn_readfirstlane(lo);
        t.rows = __builtin_amdgcn_readfirstlane(hi - lo);
        return true;
    };
    int seq = blockIdx.x / 8;
    Place now, after;
    if (!place(seq, now)) return;
    l.init();
    l.start_a(now);
    l.start_b(now);
    first_steps(l.a, l.b, lds);
    if (blockIdx.x == 0) {  // has a tile always; looks the offsets over while its first copies arrive
        bool bad = a.offsets[a.E] > a.rows;
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            bad |= a.offsets[e] < 0 || a.offsets[e + 1] < a.offsets[e];
        if (__ballot(bad) && lane_id() == 0) report(a.err, EP_DEVERR_CAPACITY);
    }
    wait_copies<0>();
    barrier_only();
    Ring ring = first_ring();
    bool behind = false;
    for (;;) {
        const bool more = place(seq += gridDim.x / 8, after);
        const NextTile<WgradLoaders<FP8>, Place> next = {l, after, more};
        f32x4 acc[MS][NS] = {};
        multiply_stream<MS, NS, F32 ? 32 : 16>(l.a, l.b, ra, rb, stream_steps<decltype(l.b)>(now.rows), lds, ring,
                                               behind, acc, next);
        const int n = now.n0 + wm * MS * 16, k = now.k0 + wn * NS * 16;
        store_block<F32, true>(a.dw, (int64_t)now.e * a.n_dim + n, k, a.k_dim, a.n_dim - n, a.k_dim - k, acc);
        if (!more) break;
        behind = now.n0 + kFullRows <= a.n_dim && now.k0 + kTileN <= a.k_dim;
        now = after;
    }
    wait_copies<0>();
}

// One workgroup per CU at most (it takes all of the CU's LDS), in multiples of
// the 8 XCDs.
template <class Args>
hipError_t launch_tiles(void (*kernel)(Args), int64_t tiles, const Args& a, hipStream_t st) {
    LaunchInfo info;
    hipError_t e = launch_info(st, reinterpret_cast<const void*>(kernel), kThreads, &info);
    if (e != hipSuccess) return e;
    const int64_t most = std::max(info.cus / 8 * 8, 8);
    // A call without rows has no tiles and only looks its offsets over.
    const unsigned grid = (unsigned)std::min(most, std::max<int64_t>(tiles + 7, 8) / 8 * 8);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

uint32_t* err_words(char* ws) { return reinterpret_cast<uint32_t*>(ws); }

}  // namespace

int64_t expert_matmul_tiles(int64_t rows, int E, int n_dim) {
    return most_tiles(rows, E, (n_dim + kTileN - 1) / kTileN);
}
int64_t expert_swiglu_tiles(int64_t rows, int E, int F) {
    return most_tiles(rows, E, (F + 127) / 128);
}
int64_t expert_wgrad_tiles(int E, int n_dim, int k_dim) {
    return (int64_t)E * ((n_dim + kFullRows - 1) / kFullRows) * ((k_dim + kTileN - 1) / kTileN);
}

hipError_t launch_expert_matmul(const ep_shape& s, const ep_layout& L, const uint16_t* x, int64_t rows, int k_dim,
                                const uint16_t* w, int n_dim, int order, uint16_t* y, char* ws, hipStream_t st) {
    const MatmulArgs a = {L.expert_offsets, x, w, y, s.E, (int)rows, k_dim, n_dim, err_words(ws)};
    return launch_tiles(order == EP_WEIGHT_KN ? matmul_kernel<true> : matmul_kernel<false>,
                        expert_matmul_tiles(rows, s.E, n_dim), a, st);
}

hipError_t launch_expert_swiglu(const ep_shape& s, const ep_layout& L, const uint16_t* x, int64_t rows,
                                const uint16_t* w13, int F, uint16_t* act, uint8_t* gu, float* scales, char* ws,
                                hipStream_t st) {
    const SwigluArgs a = {L.expert_offsets, x, w13, act, gu, scales, s.E, (int)rows, s.H, F, err_words(ws)};
    return launch_tiles(gu ? swiglu_kernel<true> : swiglu_kernel<false>, expert_swiglu_tiles(rows, s.E, F), a, st);
}

hipError_t launch_expert_wgrad(const ep_shape& s, const ep_layout& L, const uint16_t* dy, int64_t rows, int n_dim,
                               const uint16_t* x, const uint8_t* x8, const float* x_scales, int k_dim, void* dw,
                               int dtype, char* ws, hipStream_t st) {
    const WgradArgs a = {L.expert_offsets, dy, x, x8, x_scales, dw, s.E, (int)rows, n_dim, k_dim, err_words(ws)};
    void (*const kernels[2][2])(WgradArgs) = {{wgrad_kernel<false, false>, wgrad_kernel<false, true>},
                                              {wgrad_kernel<true, false>, wgrad_kernel<true, true>}};
    // Without rows the second operand may be NULL, which only the bf16 form never reads.
    return launch_tiles(kernels[x8 && rows > 0][dtype == EP_GRAD_F32], expert_wgrad_tiles(s.E, n_dim, k_dim), a, st);
}

}  // namespace ep
