// moe_gemm.cuh -- persistent grouped GEMM on the sm_100a tensor cores
// (tcgen05.mma, accumulators in TMEM, operands staged by TMA with the
// 128-byte swizzle), used for every contraction of the layer:
//   * the routed experts' gate/up projections with the SwiGLU epilogue and
//     their down projections (the "GroupGEMM" of the talk notes' Table 1 and
//     "Key findings 5"), one group per expert segment of the padded rows;
//   * the dense SwiGLU FFN (shared experts, DenseFA, DensePA) as one group;
//   * the router GEMM (fp32 logits) as one group.
//
// Orientation.  The weight rows are the MMA's M side (128 output features
// per tile) and the token rows its N side (16..kMaxN tokens per tile, a
// multiple of 16).  Decode (one or two tokens per expert) then costs a
// 128 x 16 MMA per 128 weight rows instead of a 128-row tile of padding, and
// prefill uses N up to 256.  The accumulator D[feature][token] lives in TMEM
// (lane = feature, column = token).
//
// Tiles.  A group g owns rows [seg[g], seg[g+1]) of the token matrix X.  The
// rows are cut into chunks of at most kMaxN rows (in units of 16, balanced);
// a tile is (group, 128-feature block f, chunk j), ordered f-major inside a
// group so that the chunks sharing one weight block run side by side and
// reuse it from L2.  Each tile reduces over K = kdim in steps of 128 bytes.
//
// Schedule.  gridDim.x persistent blocks (one per SM).  Whole waves of tiles
// are dealt round-robin; the remaining one to two waves (all but the first
// wave, with fewer than two) are split evenly by k-iterations across the
// blocks (stream-K), so every block streams the same
// number of weight bytes even when there are fewer tiles than SMs (decode).
// A tile split across blocks is finished by the last block to arrive: each
// contributor stores its fp32 partial tile, then increments the tile's
// counter; the block that brings the counter to the number of contributors
// sums all partials in block order (deterministic) and runs the epilogue.
// No block ever waits on another block.
//
// Roles (320 threads): warp 0 issues TMA loads, warp 1 owns TMEM and issues
// the MMAs, warps 2..9 run the epilogue (TMEM -> registers -> global), two
// warps per TMEM lane quadrant, each on half of the tile's token columns.
// Where the packed results fit in registers, the epilogue reads the whole
// accumulator, frees it for the next tile's MMAs and only then stores.  All
// waits are bounded by a deadline; a wait that runs out sets the status word
// and every role winds down (in-flight copies and MMAs are drained first).
#pragma once

#include "moe_common.cuh"

namespace moe {

constexpr int kMaxGroups = 1024;
constexpr int kGemmEpiWarps = 8;                      // two per TMEM lane quadrant
constexpr int kGemmThreads = 64 + 32 * kGemmEpiWarps;  // producer warp, MMA warp, epilogue
constexpr int kFfnThreads = 192;

// Partial-tile slot layout: column c of row r (r < 128) at float index
// ((c / 4) * 128 + r) * 4 + c % 4, so that a warp moves 32 consecutive
// float4 (512 contiguous bytes) per access.
__device__ __forceinline__ long long slot_f4(int c4, int r) { return (long long)c4 * 128 + r; }

struct GemmParams {
    const int32_t* seg_offsets;  // [n_groups + 1] row offsets into X, or nullptr: one group [0, seg_rows)
    int n_groups;
    int seg_rows;
    int n_out;            // output features
    int kdim;             // reduction length
    int w_group_stride;   // weight rows from one group to the next
    int up_offset;        // weight rows from a gate row to its up row (SwiGLU)
    void* out;            // output rows (same row index as X), out_ld elements apart
    int out_ld;
    int* counters;        // >= 2 * gridDim.x ints; zero on entry and on exit
    float* partials;      // 2 * gridDim.x slots of 128 * kAccCols floats
    unsigned* status;     // status word (bit kStatusTimeout)
    uint64_t wait_limit_ns;
    int withhold_first_load;
    int sk_min_units;     // minimum k-iterations per stream-K block
    int max_split;        // stream-K: most blocks contributing to one tile
    int split_tail;       // 1: whole waves data-parallel, the last partial wave in aligned k-slices
    int w_joined;         // MN-major weights: tm_w loads a stage's weight tiles in one copy
    int x_joined;         // stages of several k-chunks: the tm_x maps load all of them in one copy
    void* pre;            // training epilogues: pre-activations [rows, 2 n_out], gate then up columns
};

// Epilogue kinds: one 128-row weight tile per stage (plain store); gate and
// up tiles of the same 128 features (SwiGLU); two adjacent 128-feature
// blocks sharing one token tile (wide plain store, 256 features per tile).
// Training: kEpiSwiGLUTrain is the SwiGLU epilogue that also stores the
// pre-activations; kEpiSwiGLUGrad takes the accumulator as the gradient of
// the activation, reads the pre-activations (g, u) and stores the gradients
// of both: dg = dact u silu'(g), du = dact silu(g).
constexpr int kEpiPlain = 0, kEpiSwiGLU = 1, kEpiWide = 2, kEpiSwiGLUTrain = 3, kEpiSwiGLUGrad = 4;

// Weights as the MMA's M operand: rows of output features, K contiguous
// ([out, in] used forward: K-major), or for the gradients, which contract
// over the weights' out axis, rows of K with the features contiguous
// (MN-major).
template <typename T, int kEpi, int kMaxN, int kCta = 1, bool kTrainOrder = false>
struct GemmCfg {
    // Operand tiles are K-major rows of kRowBytes with the swizzle of that
    // width.  128-byte rows: 64-byte rows (twice the stages in the same
    // shared memory) measured slower on B200, the per-stage barrier and TMA
    // overhead outweighing the deeper lookahead.
    static constexpr int kRowBytes = 128;
    static constexpr int kBK = kRowBytes / Elt<T>::kBytes;  // K elements per stage
    static constexpr int kMmaK = 32 / Elt<T>::kBytes;       // K per MMA instruction
    static constexpr int kKSteps = kBK / kMmaK;             // MMAs per operand pair and stage
    static constexpr int kNW = kEpi == kEpiPlain || kEpi == kEpiSwiGLUGrad ? 1 : 2;  // weight tiles per stage
    static constexpr int kFeat = kEpi == kEpiWide ? 256 : 128;  // output features per CTA and tile
    static constexpr int kFeatTile = kFeat * kCta;                 // output features per tile
    static constexpr int kUnit = 16 * kCta;                        // token-row granularity of the MMA
    static constexpr int kWTileBytes = 128 * kRowBytes;
    static constexpr int kXBoxRows = 16;       // token rows per TMA box: 16, 64 and kMaxN
    static constexpr int kXBoxMid = 64;
    static constexpr int kXTileBytes = (kMaxN / kCta) * kRowBytes;  // this CTA's share of the token tile
    // k-chunks of kBK a stage holds, loaded in one copy per operand: two where a
    // chunk's MMAs (256 x 256 x 64 on a pair: 270 ns) take no longer than its two
    // copies' issue (65 ns each and 0.7 ns a 128-byte row)
    static constexpr int kChunks = kEpi == kEpiSwiGLUGrad ? 2 : 1;
    static constexpr int kStageK = kBK * kChunks;
    static constexpr int kWBytes = kNW * kWTileBytes * kChunks;  // a stage's weight tiles
    static constexpr int kStageBytes = kWBytes + kXTileBytes * kChunks;
    static constexpr int kAccCols = kNW * kMaxN;
    static constexpr int kNumAcc = (512 / kAccCols) >= 2 ? 2 : 1;
    // segment and chunk tables; training: the groups' order too
    static constexpr int kTableBytes = 2 * (kMaxGroups + 1) * 4 + (kTrainOrder ? kMaxGroups * 2 : 0);
    static constexpr int kMiscBytes = 512;
    static constexpr int kMaxStages = 16;
    static constexpr int kBudget = 227 * 1024 - 1024 - kTableBytes - kMiscBytes;
    static constexpr int kStagesRaw = kBudget / kStageBytes;
    static constexpr int kStages = kStagesRaw > kMaxStages ? kMaxStages : kStagesRaw;
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kTableBytes + kMiscBytes;
    static_assert(kStages >= 2, "pipeline needs two stages");
    static_assert(kMaxN % kUnit == 0 && kMaxN >= kUnit && kMaxN <= 256, "MMA N range");
    static_assert(kCta == 1 || kCta == 2, "one CTA or a CTA pair");
    static_assert(kAccCols * kNumAcc <= 512, "TMEM columns");
    static_assert(2 * kMaxStages * 8 + 2 * kNumAcc * 8 + 8 + 12 <= kMiscBytes, "barriers fit");
    static_assert(kStageBytes % 1024 == 0, "stages keep the 1024-byte alignment of the swizzle atoms");
};

// ------------------------------------------------------------- scheduling
struct Tile {
    int group, f0, row0, nrows, mma_n, wrow, nch, chunk;
};

// Two ways to share out the tiles left after the whole data-parallel waves:
//  * contiguous stream-K (split_tail 0): the last one to two waves of tiles
//    as one range of (tile, k-iteration) units cut evenly across the blocks;
//  * aligned slices (split_tail 1): every whole wave data-parallel, and the
//    tiles of the last partial wave each cut into S equal k-slices, taken
//    slice-major and dealt round-robin (block c takes units c and c + G).
//    Tiles that share a weight block (adjacent token chunks) or a token chunk
//    (feature blocks of one expert) then stream the same k-slice at the same
//    time, so the shared operand is read from DRAM once; with contiguous
//    ranges the sharing tiles sit at different k-offsets and each reads it.
struct Sched {
    int n_groups, NF, KI, G, cta;
    long long total_tiles, dp_waves, dp_tiles, sk_tiles, U;
    int G_sk;
    int S;              // aligned slices per tail tile (0: contiguous stream-K)
    // iteration state
    long long w;        // next DP wave
    long long u, u_end; // stream-K cursor
    bool sk_first;
    int next_unit;      // aligned slices: this block's next local unit (0 or 1)

    __device__ long long beg(int c) const { return (long long)c * U / G_sk; }
    // block owning stream-K unit q
    __device__ int owner(long long q) const { return (int)(((q + 1) * (long long)G_sk - 1) / U); }
};

// Slices per tail tile for the aligned split: at most 2 units per block (the
// two partial slots), at least min_units k-iterations per slice, at most
// max_split contributors per tile; among those, the fewest slices with the
// shortest tail, ceil(tail * S / G) / S tile-times.
__device__ __forceinline__ int aligned_slices(long long tail, int G, int KI, long long min_units, int max_split) {
    if (tail <= 0) return 1;
    long long smax = (2LL * G) / tail;
    if (smax > max_split) smax = max_split;
    if (smax > KI / min_units) smax = KI / min_units;
    int best = 1;
    double best_t = (double)((tail + G - 1) / G);
    for (int s = 2; s <= smax; ++s) {
        const double t = (double)((tail * s + G - 1) / G) / s;
        if (t < best_t - 1e-9) {
            best_t = t;
            best = s;
        }
    }
    return best;
}

struct Item {
    long long tile;
    int kb, ke;
    bool split;   // partial tile (stream-K fixup)
    int slot;     // partial slot of this block (0 or 1)
    long long sk_tile;
};

// Scheduling unit: one CTA, or one CTA pair (cluster of 2) sharing each tile.
__device__ __forceinline__ void sched_init(Sched& s, const GemmParams& p, int total_chunks, int NF, int KI, int ncta) {
    s.n_groups = p.n_groups;
    s.NF = NF;
    s.KI = KI;
    s.G = gridDim.x / ncta;
    s.cta = blockIdx.x / ncta;
    s.total_tiles = (long long)total_chunks * NF;
    // at most max_split blocks share one tile: every block takes >= KI / kMaxSplit k-iterations
    long long min_units = (KI + p.max_split - 1) / p.max_split;
    if (min_units < p.sk_min_units) min_units = p.sk_min_units;
    s.S = 0;
    s.next_unit = 0;
    if (p.split_tail) {
        s.dp_waves = s.total_tiles / s.G;
        s.dp_tiles = s.dp_waves * s.G;
        s.sk_tiles = s.total_tiles - s.dp_tiles;  // < G: fits the counters and two slots per block
        s.S = aligned_slices(s.sk_tiles, s.G, KI, min_units, p.max_split);
        s.U = 0;
        s.G_sk = s.G;
        s.w = 0;
        s.u = s.u_end = 0;
        s.sk_first = true;
        return;
    }
    // Whole waves first, keeping one to two waves for the stream-K tail; with
    // fewer than two waves of tiles, one whole wave and the rest as stream-K,
    // so that the token chunks sharing a weight block (adjacent tiles) stream
    // it together at least in that wave.
    s.dp_waves = s.total_tiles >= 2LL * s.G ? s.total_tiles / s.G - 1 : (s.total_tiles >= s.G ? 1 : 0);
    s.dp_tiles = s.dp_waves * s.G;
    s.sk_tiles = s.total_tiles - s.dp_tiles;
    s.U = s.sk_tiles * KI;
    long long gsk = s.U / min_units;
    if (gsk < 1) gsk = 1;
    if (gsk > s.G) gsk = s.G;
    s.G_sk = (int)gsk;
    s.w = 0;
    if (s.U > 0 && s.cta < s.G_sk) {
        s.u = s.beg(s.cta);
        s.u_end = s.beg(s.cta + 1);
    } else {
        s.u = s.u_end = 0;
    }
    s.sk_first = true;
}

// kMixed (training): the groups come by descending tokens per tile, so a tile
// of many tokens, bound by its MMAs, stands at the front and one of few, bound
// by reading its weights, at the back.  The whole waves are dealt back and
// forth, which evens out the blocks' sums, and each block takes its tiles
// alternately from both ends, one half of the blocks starting at the front and
// the other at the back: the MMAs of the one kind then run under the reads of
// the other.
template <bool kMixed>
__device__ __forceinline__ bool sched_next(Sched& s, Item& it) {
    if (s.w < s.dp_waves) {
        if (kMixed) {
            const bool front = ((s.w & 1) == 0) == (s.cta < s.G / 2);
            const long long wave = front ? s.w / 2 : s.dp_waves - 1 - s.w / 2;
            it.tile = wave * s.G + ((wave & 1) ? s.G - 1 - s.cta : s.cta);
        } else {
            it.tile = s.w * s.G + s.cta;
        }
        it.kb = 0;
        it.ke = s.KI;
        it.split = false;
        it.slot = 0;
        it.sk_tile = -1;
        ++s.w;
        return true;
    }
    if (s.u < s.u_end) {
        long long st = s.u / s.KI;
        int kb = (int)(s.u - st * s.KI);
        long long left = s.u_end - s.u;
        int ke = (int)((long long)kb + left < s.KI ? kb + left : s.KI);
        it.tile = s.dp_tiles + st;
        it.kb = kb;
        it.ke = ke;
        it.sk_tile = st;
        it.split = !(kb == 0 && ke == s.KI);
        it.slot = s.sk_first ? 0 : 1;
        s.sk_first = false;
        s.u += ke - kb;
        return true;
    }
    if (s.S > 0 && s.next_unit < 2) {
        // aligned slices: unit q = cta + j G is slice q / tail of tail tile q % tail
        const long long q = (long long)s.cta + (long long)s.next_unit * s.G;
        if (q >= s.sk_tiles * s.S) return false;
        const long long st = q % s.sk_tiles;
        const int sl = (int)(q / s.sk_tiles);
        it.tile = s.dp_tiles + st;
        it.kb = (int)((long long)sl * s.KI / s.S);
        it.ke = (int)((long long)(sl + 1) * s.KI / s.S);
        it.sk_tile = st;
        it.split = s.S > 1;
        it.slot = s.next_unit;
        ++s.next_unit;
        return true;
    }
    return false;
}

// Rows of chunk j of a group of `rows` rows cut into `nch` chunks, in units of `unit` rows.
__device__ __forceinline__ void chunk_rows(int rows, int nch, int j, int unit, int& start, int& n, int& mma_n) {
    int units = (rows + unit - 1) / unit;
    int base = units / nch, extra = units % nch;
    int su = j * base + (j < extra ? j : extra);
    int mu = base + (j < extra ? 1 : 0);
    start = su * unit;
    mma_n = mu * unit;
    int left = rows - start;
    n = mma_n < left ? mma_n : left;
}

__device__ __forceinline__ int chunks_of(int rows, int max_n, int unit) {
    if (rows <= 0) return 0;
    int units = (rows + unit - 1) / unit;
    int per = max_n / unit;
    return (units + per - 1) / per;
}

// `order` (nullable): cbase runs over the groups in that order.
__device__ __forceinline__ Tile decode_tile_w(long long tile, const int* seg, const int* cbase, int n_groups, int NF,
                                              int feat, int unit, int w_group_stride,
                                              const uint16_t* order = nullptr) {
    // group: largest g with cbase[g] * NF <= tile
    int lo = 0, hi = n_groups - 1;
    while (lo < hi) {
        int mid = (lo + hi + 1) >> 1;
        if ((long long)cbase[mid] * NF <= tile) lo = mid;
        else hi = mid - 1;
    }
    int g = lo;
    int nch = cbase[g + 1] - cbase[g];
    long long local = tile - (long long)cbase[g] * NF;
    int f = (int)(local / nch);
    int j = (int)(local - (long long)f * nch);
    Tile t;
    const int first_chunk = cbase[g];
    if (order) g = order[g];
    int start, n, mn;
    chunk_rows(seg[g + 1] - seg[g], nch, j, unit, start, n, mn);
    t.group = g;
    t.f0 = f * feat;
    t.row0 = seg[g] + start;
    t.nrows = n;
    t.mma_n = mn;
    t.wrow = g * w_group_stride + f * feat;
    t.nch = nch;
    t.chunk = first_chunk + j;
    return t;
}

__device__ __forceinline__ Tile decode_tile(long long tile, const int* seg, const int* cbase, int n_groups, int NF,
                                            int feat, int unit, const GemmParams& p,
                                            const uint16_t* order = nullptr) {
    return decode_tile_w(tile, seg, cbase, n_groups, NF, feat, unit, p.w_group_stride, order);
}

template <typename OutT>
__device__ __forceinline__ void store_out(OutT* ptr, float v);
template <>
__device__ __forceinline__ void store_out<float>(float* ptr, float v) { *ptr = v; }
template <>
__device__ __forceinline__ void store_out<__half>(__half* ptr, float v) {
    *ptr = __float2half_rn(v);
}
template <>
__device__ __forceinline__ void store_out<__nv_bfloat16>(__nv_bfloat16* ptr, float v) {
    *ptr = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// ------------------------------------------------------------------ kernel
template <typename T, typename OutT, int kEpi, int kMaxN, int kCta, bool kWMn = false>
__global__ void __launch_bounds__(kGemmThreads, 1)
    moe_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ CUtensorMap tm_x64, const __grid_constant__ CUtensorMap tm_xbig,
                    const GemmParams p) {
    constexpr bool kTrain = kWMn || kEpi == kEpiSwiGLUTrain;
    using C = GemmCfg<T, kEpi, kMaxN, kCta, kTrain>;
    constexpr bool kSwiGLU = kEpi == kEpiSwiGLU || kEpi == kEpiSwiGLUTrain;
    static_assert(!kWMn || (kCta == 2 && Elt<T>::kBytes == 2 && C::kBK == 64), "MN-major weights: 16-bit, on pairs");
    static_assert(C::kChunks == 1 || kWMn, "stages of several k-chunks: MN-major weights");
    constexpr bool kTwo = C::kNW == 2;
    constexpr bool kPair = kCta == 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stage_base = smem;
    int* seg = reinterpret_cast<int*>(smem + C::kStages * C::kStageBytes);
    int* cbase = seg + (kMaxGroups + 1);
    uint16_t* order = kTrain ? reinterpret_cast<uint16_t*>(cbase + (kMaxGroups + 1)) : nullptr;
    uint8_t* misc = reinterpret_cast<uint8_t*>(cbase + (kMaxGroups + 1)) + (kTrain ? kMaxGroups * 2 : 0);
    uint64_t* full = reinterpret_cast<uint64_t*>(misc);
    uint64_t* empty = full + C::kStages;
    uint64_t* tfull = empty + C::kStages;
    uint64_t* tempty = tfull + C::kNumAcc;
    uint64_t* drain_bar = tempty + C::kNumAcc;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int* bcast = const_cast<int*>(abort_flag) + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int n_groups = p.n_groups;
    const uint64_t deadline = p.wait_limit_ns;  // per-wait limit
    // CTA pair: rank 0 (the leader) issues the MMAs for both; each CTA stages
    // its own 128 weight rows and half of the token rows, and holds in TMEM
    // the accumulators of its own 128 weight rows.
    const uint32_t rank = kPair ? cluster_rank() : 0u;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < C::kNumAcc; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], kGemmEpiWarps * kCta);
        }
        mbar_init(drain_bar, 1);
        fence_barrier_init();
        *abort_flag = 0;
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_x64);
        tma_prefetch_desc(&tm_xbig);
    }
    if (warp == 1) {
        if (kPair) tmem_alloc_pair(tmem_holder, 512);
        else tmem_alloc(tmem_holder, 512);
    }
    if (kPair) cluster_sync_all();  // the peer's barriers are initialised before any TMA or commit targets them
    pdl_wait();  // everything below reads or writes data shared with earlier kernels
    // segment table
    for (int g = threadIdx.x; g <= n_groups; g += blockDim.x)
        seg[g] = p.seg_offsets ? p.seg_offsets[g] : (g == 0 ? 0 : p.seg_rows);
    __syncthreads();
    if constexpr (kTrain) {
        // groups by descending tokens per tile, the lower index first among equals
        auto per_tile = [&](int g) {
            const int rows = seg[g + 1] - seg[g], n = chunks_of(rows, kMaxN, C::kUnit);
            return n > 0 ? (rows + n - 1) / n : 0;
        };
        int* key = cbase;  // not in use yet
        for (int g = threadIdx.x; g < n_groups; g += blockDim.x) key[g] = per_tile(g);
        __syncthreads();
        for (int g = threadIdx.x; g < n_groups; g += blockDim.x) {
            const int mine = key[g];
            int place = 0;
            for (int o = 0; o < n_groups; ++o) place += key[o] > mine || (key[o] == mine && o < g);
            order[place] = (uint16_t)g;
        }
        __syncthreads();
    }
    if (warp == 0) {
        int running = 0;
        for (int base = 0; base < n_groups; base += 32) {
            int g = base + lane;
            int n = 0;
            if (g < n_groups) {
                const int o = kTrain ? order[g] : g;
                n = chunks_of(seg[o + 1] - seg[o], kMaxN, C::kUnit);
            }
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (g < n_groups) cbase[g] = running + incl - n;
            running += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) cbase[n_groups] = running;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    const int NF = (p.n_out + C::kFeatTile - 1) / C::kFeatTile;
    const int KI = (p.kdim + C::kStageK - 1) / C::kStageK;
    Sched sch;
    sched_init(sch, p, cbase[n_groups], NF, KI, kCta);

    // training: rows of the box that holds a CTA's xn token rows
    auto x_box = [](int xn) {
        return xn <= C::kXBoxRows ? C::kXBoxRows : xn <= C::kXBoxMid ? C::kXBoxMid : kMaxN / kCta;
    };
    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (lane == 0) {
            // weights read by one tile only are streamed with evict-first; weight
            // blocks that several token chunks share stay at normal priority
            const uint64_t pol_w_once = policy_evict_first();
            const uint64_t pol_w_shared = policy_evict_normal();
            const uint64_t pol_x = policy_evict_last();
            int fills[C::kStages];
#pragma unroll
            for (int s = 0; s < C::kStages; ++s) fills[s] = 0;
            uint32_t kc = 0;
            bool withhold = p.withhold_first_load && blockIdx.x == 0;
            bool ok = true;
            Item it;
            while (ok && sched_next<kTrain>(sch, it)) {
                Tile t = decode_tile(it.tile, seg, cbase, n_groups, NF, C::kFeatTile, C::kUnit, p, order);
                // this CTA's weight rows and token rows of the tile
                const int wrow = t.wrow + (int)rank * C::kFeat;
                const int xn = t.mma_n / kCta;
                const int xrow = t.row0 + (int)rank * xn;
                // Training variants load the token rows as one box, the smallest of the
                // three that holds them (rows past the chunk are not multiplied): the
                // issuing thread takes 50-90 ns per copy, which at two to four boxes a
                // stage is longer than the stage's MMAs (256 x 256 x 64: 270 ns).
                const int xl = kTrain ? x_box(xn) : xn;
                // bytes landing on the (leader's) full barrier per stage: both CTAs' shares
                const uint32_t bytes = kCta * (C::kWBytes + C::kChunks * xl * C::kRowBytes);
                const uint64_t pol_w = t.nch > 1 ? pol_w_shared : pol_w_once;
                for (int k = it.kb; k < it.ke; ++k, ++kc) {
                    const int s = kc % C::kStages;
                    const uint32_t ph = (kc / C::kStages) & 1u;
                    if (!mbar_wait_bounded(&empty[s], ph ^ 1u, deadline, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (withhold) {  // test hook: this stage is never filled
                        withhold = false;
                        continue;
                    }
                    uint8_t* st = stage_base + s * C::kStageBytes;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                    const uint32_t fb = kPair ? map_to_rank(smem_u32(&full[s]), 0) : 0u;
                    auto load = [&](void* dst, const CUtensorMap* m, int c1, uint64_t pol) {
                        if (kPair) tma_load_2d_pair(dst, m, fb, k * C::kBK, c1, pol);
                        else tma_load_2d(dst, m, &full[s], k * C::kBK, c1, pol);
                    };
                    if constexpr (kWMn) {
                        // boxes of 64 features by kStageK rows of K; K rows past kdim read as zero
                        const int f0 = t.f0 + (int)rank * C::kFeat;
                        if (p.w_joined)
                            tma_load_4d_pair(st, &tm_w, fb, 0, k * C::kStageK, f0 / 64, t.group, pol_w);
                        else
#pragma unroll
                            for (int b = 0; b < 2 * C::kNW; ++b)
                                tma_load_3d_pair(st + b * (C::kStageK * 128), &tm_w, fb, f0 + 64 * b, k * C::kStageK,
                                                 t.group, pol_w);
                    } else {
                        load(st, &tm_w, wrow, pol_w);
                        if (kTwo) load(st + C::kWTileBytes, &tm_w, wrow + (kSwiGLU ? p.up_offset : 128), pol_w);
                    }
                    uint8_t* xs = st + C::kWBytes;
                    if constexpr (C::kChunks > 1) {
                        const CUtensorMap* m = xl == C::kXBoxRows ? &tm_x : xl == C::kXBoxMid ? &tm_x64 : &tm_xbig;
                        if (p.x_joined)
                            tma_load_4d_pair(xs, m, fb, 0, xrow, k * C::kChunks, 0, pol_x);
                        else
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_2d_pair(xs + c * xl * C::kRowBytes, m, fb, k * C::kStageK + c * C::kBK, xrow,
                                                 pol_x);
                        ++fills[s];
                        continue;
                    }
                    int r = 0;
                    if (kMaxN / kCta > C::kXBoxMid && xl == kMaxN / kCta) {
                        load(xs, &tm_xbig, xrow, pol_x);
                        r = xl;
                    }
                    if (kMaxN / kCta >= C::kXBoxMid)
                        for (; r + C::kXBoxMid <= xl; r += C::kXBoxMid)
                            load(xs + r * C::kRowBytes, &tm_x64, xrow + r, pol_x);
                    for (; r < xl; r += C::kXBoxRows) load(xs + r * C::kRowBytes, &tm_x, xrow + r, pol_x);
                    ++fills[s];
                }
            }
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.status, kStatusTimeout);
            }
            // every issued copy lands before the block exits (the leader's full
            // barriers count both CTAs' copies; the pair leaves together)
            if (rank == 0)
                for (int s = 0; s < C::kStages; ++s)
                    if (fills[s] > 0) mbar_drain(&full[s], (uint32_t)(fills[s] - 1) & 1u, p.wait_limit_ns);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0 && rank == 0) {
            // One thread issues a stage's MMAs and its commit in the time the
            // tensor core takes for them (a pair's 256 x 256 x 64 step: 512
            // cycles), so the stage cursor and the descriptors are kept
            // incrementally and one commit frees the stage in both CTAs:
            // recomputing them and committing twice took 705 cycles a step.
            uint32_t ac = 0, s = 0, ph = 0;
            bool ok = true;
            Item it;
            auto desc = [](uint32_t a) { return C::kRowBytes == 128 ? umma_desc_sw128(a) : umma_desc_sw64(a); };
            auto wdesc = [desc](uint32_t a) { return kWMn ? umma_desc_mn_sw128<C::kStageK>(a) : desc(a); };
            // K of one MMA: 32 bytes along a K-major row, 16 rows of 128 bytes in an MN-major box
            constexpr uint32_t kWStep = kWMn ? 16 * 128 / 16 : 2;
            const uint64_t w_base = wdesc(smem_u32(stage_base));
            const uint64_t x_base = desc(smem_u32(stage_base + C::kWBytes));
            while (ok && sched_next<kTrain>(sch, it)) {
                Tile t = decode_tile(it.tile, seg, cbase, n_groups, NF, C::kFeatTile, C::kUnit, p, order);
                const int b = ac % C::kNumAcc;
                const uint32_t aph = (ac / C::kNumAcc) & 1u;
                if (!mbar_wait_bounded(&tempty[b], aph ^ 1u, deadline, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_gate = tmem_base + b * C::kAccCols;
                const uint32_t d_up = d_gate + kMaxN;
                const uint32_t idesc = umma_idesc(Elt<T>::kMmaFmt, 128 * kCta, t.mma_n) | (kWMn ? kIdescAMn : 0u);
                uint32_t acc = 0;
                // from one k-chunk of the token rows to the next
                const uint32_t x_chunk = C::kChunks > 1 ? (uint32_t)(x_box(t.mma_n / kCta) * C::kRowBytes) >> 4 : 0u;
                for (int k = it.kb; k < it.ke; ++k) {
                    if (!mbar_wait_bounded(&full[s], ph, deadline, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a0 = w_base + s * (C::kStageBytes >> 4);
                    const uint64_t a1 = a0 + (C::kWTileBytes >> 4);
                    const uint64_t bx = x_base + s * (C::kStageBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < C::kKSteps * C::kChunks; ++kk) {
                        const uint32_t ac_kk = kk > 0 ? 1u : acc;
                        const uint64_t b = bx + (kk / C::kKSteps) * x_chunk + 2 * (kk % C::kKSteps);
                        if (kPair) {
                            umma_pair_bf16(d_gate, a0 + kWStep * kk, b, idesc, ac_kk);
                            if (kTwo) umma_pair_bf16(d_up, a1 + kWStep * kk, b, idesc, ac_kk);
                        } else {
                            umma<T>(d_gate, a0 + kWStep * kk, b, idesc, ac_kk);
                            if (kTwo) umma<T>(d_up, a1 + kWStep * kk, b, idesc, ac_kk);
                        }
                    }
                    acc = 1;
                    if (kPair) umma_commit_pair_both(&empty[s]);  // the stage is free in both CTAs
                    else umma_commit(&empty[s]);
                    if (++s == C::kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                if (kPair) umma_commit_pair_both(&tfull[b]);
                else umma_commit(&tfull[b]);
                ++ac;
            }
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.status, kStatusTimeout);
                if (kPair) umma_commit_pair(smem_u32(drain_bar));
                else umma_commit(drain_bar);
                mbar_drain(drain_bar, 0, p.wait_limit_ns);
            }
        }
    } else {
        // -------------------------------------------------------- epilogue
        const int quad = warp & 3;                // TMEM lane quadrant this warp may access
        const int half = (warp - 2) >> 2;         // which share of the token columns
        const int r = quad * 32 + lane;           // TMEM lane = feature row within a 128-row block
        const int e = (warp - 2) * 32 + lane;     // epilogue thread 0 .. 255
        constexpr int kEpiThreads = 32 * kGemmEpiWarps;
        constexpr int kHalfN = kMaxN / (kGemmEpiWarps / 4);  // token columns per warp
        constexpr int kCh = kHalfN >= 32 && kEpi != kEpiSwiGLUGrad ? 32 : 16;
        constexpr bool kBf16Out = sizeof(OutT) == 2;
        constexpr int kRegs = kBf16Out ? kHalfN / 2 : kHalfN;  // packed results of one accumulator
        constexpr bool kEarly = (kEpi == kEpiPlain || kEpi == kEpiSwiGLU) && kRegs <= 64;
        OutT* out = reinterpret_cast<OutT*>(p.out);
        uint32_t ac = 0;
        Item it;
        while (sched_next<kTrain>(sch, it)) {
            Tile t = decode_tile(it.tile, seg, cbase, n_groups, NF, C::kFeatTile, C::kUnit, p, order);
            const int b = ac % C::kNumAcc;
            const uint32_t aph = (ac / C::kNumAcc) & 1u;
            // this warp's token columns: half of the accumulator's, or (training,
            // where chunks are often short of it) half of the tile's
            const int share = kTrain ? (t.mma_n / 2 + 15) / 16 * 16 : kHalfN;
            const int cbeg = half * share;
            const int cend = t.nrows < cbeg + share ? t.nrows : cbeg + share;  // this half's real columns
            // kEpiSwiGLUGrad: this lane's feature of 16 tokens' pre-activations, gate
            // and up, requested one block ahead of their use (a tile's first before
            // its MMAs are waited for); loaded where they were used, they held a tile
            // up for 80 us, where its MMAs at K = 4096 take 18 us
            uint16_t pre[kEpi == kEpiSwiGLUGrad ? 32 : 1];
            const uint16_t* pre_in = nullptr;
            if constexpr (kEpi == kEpiSwiGLUGrad) {
                const int pf = t.f0 + (int)rank * C::kFeat + r;
                if (pf < p.n_out) pre_in = reinterpret_cast<const uint16_t*>(p.pre) + (long long)t.row0 * 2 * p.n_out + pf;
            }
            auto pre_fetch = [&](int c0) {
                if constexpr (kEpi == kEpiSwiGLUGrad) {
                    if (!pre_in) return;
                    const uint16_t* q = pre_in + (long long)c0 * 2 * p.n_out;
                    auto get = [&](int i) {
                        pre[i] = *q;
                        q += p.n_out;
                        pre[16 + i] = *q;
                        q += p.n_out;
                    };
                    if (c0 + 16 <= cend) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) get(i);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c0 + i < cend) get(i);
                    }
                }
            };
            if (!it.split) pre_fetch(cbeg);  // a split tile: only the block that finishes it reads them
            // every epilogue thread goes on, or all leave (the split path below
            // meets at named barriers, which a thread that left would never reach)
            const bool got = mbar_wait_bounded(&tfull[b], aph, deadline, abort_flag);
            if (!named_all(1, kEpiThreads, got)) {
                *abort_flag = 1;
                atomicOr(p.status, kStatusTimeout);
                break;
            }
            tc_fence_after();
            const uint32_t tacc = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + b * C::kAccCols;
            const int f = t.f0 + (int)rank * C::kFeat + r;
            // valid rows of the first and second accumulator
            const bool v0 = f < p.n_out;
            const bool v1 = kEpi == kEpiWide ? (f + 128 < p.n_out) : (kSwiGLU && v0);
            OutT* orow = out + (long long)t.row0 * p.out_ld + f;
            // kCh columns of the first (and second) accumulator from column c0, one wait
            auto load_cols = [&](int c0, float (&g)[kCh], float (&u)[kCh]) {
                uint32_t ga[kCh], ua[kCh];
                if constexpr (kCh == 32) {
                    tmem_ld32_nowait(tacc + c0, ga);
                    if (kTwo) tmem_ld32_nowait(tacc + kMaxN + c0, ua);
                } else {
                    tmem_ld16_nowait(tacc + c0, ga);
                    if (kTwo) tmem_ld16_nowait(tacc + kMaxN + c0, ua);
                }
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < kCh; ++i) {
                    g[i] = __uint_as_float(ga[i]);
                    u[i] = kTwo ? __uint_as_float(ua[i]) : 0.f;
                }
            };
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();  // one arrival per warp
                if (lane == 0) {
                    if (kPair && rank != 0) mbar_arrive_cluster(map_to_rank(smem_u32(&tempty[b]), 0));
                    else mbar_arrive(&tempty[b]);
                }
            };
            // g: first accumulator, u: second (up projection, or features f + 128)
            const int nrows = t.nrows;
            const long long out_ld = p.out_ld;
            // (callers skip blocks that start past the last real column; whole
            // blocks store without per-element predicates, which measured
            // markedly faster than predicating every store)
            OutT* prow = nullptr;  // this feature's pre-activation column (training)
            if constexpr (kEpi == kEpiSwiGLUTrain || kEpi == kEpiSwiGLUGrad)
                prow = reinterpret_cast<OutT*>(p.pre) + (long long)t.row0 * 2 * p.n_out + f;
            const int n_out = p.n_out;
            auto emit = [orow, prow, n_out, nrows, out_ld, v0, v1, &pre, &pre_fetch](int c0, float (&g)[16], float (&u)[16]) {
                const int n = nrows - c0 < 16 ? nrows - c0 : 16;
                if constexpr (kEpi == kEpiSwiGLUTrain) {
                    // pointers step from row to row: an address computed for each store
                    // cost more than the store (8 experts of 256 rows x 128 x 128: 14.1
                    // us, 11.8 us)
                    OutT* pr = prow + (long long)c0 * 2 * n_out;
                    OutT* act = orow + c0 * out_ld;
                    auto put = [&](int i) {
                        store_out<OutT>(pr, g[i]);
                        pr += n_out;
                        store_out<OutT>(pr, u[i]);
                        pr += n_out;
                        store_out<OutT>(act, silu_mul(g[i], u[i]));
                        act += n_out;
                    };
                    if (v0 && n == 16) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) put(i);
                    } else if (v0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < n) put(i);
                    }
                    return;
                }
                if constexpr (kEpi == kEpiSwiGLUGrad) {
                    float pg[16], pu[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        pg[i] = __uint_as_float((uint32_t)pre[i] << 16);
                        pu[i] = __uint_as_float((uint32_t)pre[16 + i] << 16);
                    }
                    pre_fetch(c0 + 16);
                    OutT* o = orow + c0 * out_ld;
                    auto put = [&](int i) {
                        const float sg = __fdividef(1.f, 1.f + __expf(-pg[i]));
                        store_out<OutT>(o, g[i] * pu[i] * sg * (1.f + pg[i] * (1.f - sg)));
                        o += n_out;
                        store_out<OutT>(o, g[i] * pg[i] * sg);
                        o += n_out;
                    };
                    if (v0 && n == 16) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) put(i);
                    } else if (v0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < n) put(i);
                    }
                    return;
                }
                if (n == 16) {
                    if (v0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) store_out<OutT>(orow + (c0 + i) * out_ld, g[i]);
                    }
                    if (kEpi == kEpiWide && v1) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) store_out<OutT>(orow + 128 + (c0 + i) * out_ld, u[i]);
                    }
                } else {
                    if (v0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < n) store_out<OutT>(orow + (c0 + i) * out_ld, g[i]);
                    }
                    if (kEpi == kEpiWide && v1) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < n) store_out<OutT>(orow + 128 + (c0 + i) * out_ld, u[i]);
                    }
                }
            };
            if (!it.split && kEarly) {
                // whole half into registers (SwiGLU applied, packed), accumulator freed, then stores
                uint32_t res[kRegs];
#pragma unroll
                for (int j = 0; j < kHalfN / kCh; ++j) {
                    const int c0 = cbeg + j * kCh;
                    if (c0 < cend) {
                        float g[kCh], u[kCh];
                        load_cols(c0, g, u);
#pragma unroll
                        for (int i = 0; i < kCh; ++i)
                            if (kSwiGLU) g[i] = silu_mul(g[i], u[i]);
                        if constexpr (kBf16Out) {
#pragma unroll
                            for (int i = 0; i < kCh; i += 2) {
                                __nv_bfloat162 h2 = __floats2bfloat162_rn(g[i], g[i + 1]);
                                res[(j * kCh + i) / 2] = *reinterpret_cast<uint32_t*>(&h2);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < kCh; ++i) res[j * kCh + i] = __float_as_uint(g[i]);
                        }
                    }
                }
                release();
                // column i of this warp's share from the packed registers
                auto store_res = [&](int i) {
                    OutT* dst = orow + (long long)(cbeg + i) * out_ld;
                    if constexpr (kBf16Out) {
                        const uint32_t w2 = res[i / 2];
                        *reinterpret_cast<uint16_t*>(dst) = (i & 1) ? (uint16_t)(w2 >> 16) : (uint16_t)(w2 & 0xffffu);
                    } else {
                        *reinterpret_cast<float*>(dst) = __uint_as_float(res[i]);
                    }
                };
                if (v0) {
#pragma unroll
                    for (int j = 0; j < kHalfN / 16; ++j) {
                        const int c0 = cbeg + 16 * j;
                        if (c0 + 16 <= cend) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) store_res(16 * j + i);
                        } else if (c0 < cend) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (c0 + i < cend) store_res(16 * j + i);
                        }
                    }
                }
            } else if (!it.split) {
                // kCh columns of both accumulators per TMEM round trip, stored 16 at a time
                for (int c0 = cbeg; c0 < cend; c0 += kCh) {
                    uint32_t ga[kCh], ua[kCh];
                    if constexpr (kCh == 32) {
                        tmem_ld32_nowait(tacc + c0, ga);
                        if (kTwo) tmem_ld32_nowait(tacc + kMaxN + c0, ua);
                    } else {
                        tmem_ld16_nowait(tacc + c0, ga);
                        if (kTwo) tmem_ld16_nowait(tacc + kMaxN + c0, ua);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < kCh / 16; ++h) {
                        float g[16], u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            g[i] = __uint_as_float(ga[16 * h + i]);
                            u[i] = kTwo ? __uint_as_float(ua[16 * h + i]) : 0.f;
                            if (kEpi == kEpiSwiGLU) g[i] = silu_mul(g[i], u[i]);
                        }
                        if (c0 + 16 * h < cend) emit(c0 + 16 * h, g, u);
                    }
                }
                release();
            } else {
                // stream-K: publish this block's partial tile (rows of real
                // output features and columns of real tokens only)
                const long long slot_floats = 128LL * C::kAccCols;
                float4* mine = reinterpret_cast<float4*>(p.partials + ((long long)blockIdx.x * 2 + it.slot) * slot_floats);
                const long long counter = it.sk_tile * kCta + rank;  // one counter per tile half
                for (int c0 = cbeg; c0 < cend; c0 += kCh) {
                    float g[kCh], u[kCh];
                    load_cols(c0, g, u);
                    if (v0) {
#pragma unroll
                        for (int q = 0; q < kCh / 4; ++q)
                            mine[slot_f4((c0 >> 2) + q, r)] =
                                make_float4(g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]);
                    }
                    if (kTwo && v1) {
#pragma unroll
                        for (int q = 0; q < kCh / 4; ++q)
                            mine[slot_f4(((kMaxN + c0) >> 2) + q, r)] =
                                make_float4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
                    }
                }
                named_sync(1, kEpiThreads);
                if (e == 0) *bcast = atomic_add_acq_rel_gpu(&p.counters[counter], 1);
                named_sync(1, kEpiThreads);
                const int arrived = *bcast;
                // contributors: blocks whose stream-K range meets this tile, or
                // (aligned slices) the S slices' units
                const bool aligned = sch.S > 0;
                const long long q0 = it.sk_tile * sch.KI;
                const int c_first = aligned ? 0 : sch.owner(q0);
                const int c_last = aligned ? sch.S - 1 : sch.owner(q0 + sch.KI - 1);
                int ncontrib = 0;
                if (aligned) {
                    ncontrib = sch.S;
                } else {
                    for (int c = c_first; c <= c_last; ++c)
                        if (sch.beg(c) < sch.beg(c + 1)) ++ncontrib;
                }
                if (arrived == ncontrib - 1) {
                    // last to arrive: sum every contribution in block order, then the epilogue
                    pre_fetch(cbeg);
                    for (int c0 = cbeg; c0 < cend; c0 += 16) {
                        float g[16], u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) g[i] = u[i] = 0.f;
                        for (int i = c_first; i <= c_last; ++i) {
                            // contributor i: a block (contiguous) or a slice (aligned), in k order
                            int c, slot;
                            if (aligned) {
                                // at most two slices a block (aligned_slices): no division
                                const long long q = it.sk_tile + (long long)i * sch.sk_tiles;
                                slot = q >= sch.G;
                                c = (int)(q - (slot ? sch.G : 0));
                            } else {
                                c = i;
                                const long long bc = sch.beg(c);
                                if (bc >= sch.beg(c + 1)) continue;
                                slot = (bc / sch.KI == it.sk_tile) ? 0 : 1;
                            }
                            if (c == sch.cta && slot == it.slot) {
                                uint32_t va[16], vb[16];
                                tmem_ld16_nowait(tacc + c0, va);
                                if (kTwo) tmem_ld16_nowait(tacc + kMaxN + c0, vb);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    g[i] += __uint_as_float(va[i]);
                                    if (kTwo) u[i] += __uint_as_float(vb[i]);
                                }
                            } else {
                                const float4* other =
                                    reinterpret_cast<const float4*>(p.partials + (((long long)c * kCta + rank) * 2 + slot) *
                                                                                     slot_floats);
                                const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                                float4 a4[4], b4[4];
#pragma unroll
                                for (int q = 0; q < 4; ++q) a4[q] = v0 ? __ldcg(other + slot_f4((c0 >> 2) + q, r)) : z;
                                if (kTwo) {
#pragma unroll
                                    for (int q = 0; q < 4; ++q)
                                        b4[q] = v1 ? __ldcg(other + slot_f4(((kMaxN + c0) >> 2) + q, r)) : z;
                                }
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    g[4 * q] += a4[q].x;
                                    g[4 * q + 1] += a4[q].y;
                                    g[4 * q + 2] += a4[q].z;
                                    g[4 * q + 3] += a4[q].w;
                                }
                                if (kTwo) {
#pragma unroll
                                    for (int q = 0; q < 4; ++q) {
                                        u[4 * q] += b4[q].x;
                                        u[4 * q + 1] += b4[q].y;
                                        u[4 * q + 2] += b4[q].z;
                                        u[4 * q + 3] += b4[q].w;
                                    }
                                }
                            }
                        }
                        if (kEpi == kEpiSwiGLU) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) g[i] = silu_mul(g[i], u[i]);
                        }
                        emit(c0, g, u);
                    }
                    if (e == 0) p.counters[counter] = 0;  // leave the counter zero for the next launch
                }
                release();
            }
            ++ac;
        }
    }

    tc_fence_before();
    if (kPair) cluster_sync_all();  // neither CTA frees TMEM or leaves while the pair's MMAs may run
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (kPair) tmem_dealloc_pair(tmem_base, 512);
        else tmem_dealloc(tmem_base, 512);
    }
}

}  // namespace moe
