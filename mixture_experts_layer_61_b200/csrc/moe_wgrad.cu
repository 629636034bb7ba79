// moe_wgrad.cu -- weight gradients of the experts' products on the sm_100a
// tensor cores: for every expert e, over the rows p of its segment,
//   out[e] [m, n] = sum_p d[p, m] x[p, n]
// (dW2 with d the gradient of the down projection's output and x the
// activations; dW13 with d the gradients of the pre-activations and x the
// permuted tokens).  The reduction runs over the rows, so both operands are
// taken MN-major, as they lie in memory: a TMA box is 64 columns by 64 rows.
//
// A CTA pair computes a 256 x 256 tile with the 2-SM MMA (each CTA stages its
// 128 columns of d and half of the 256 columns of x: 32 KB for 64 rows, 512
// cycles of MMA), two accumulators in TMEM so that the epilogue of one tile
// runs under the MMAs of the next: with a few hundred rows per expert a tile
// has only a handful of k-steps and its 128 KB of output weighs as much as its
// operands.  Reads from L2 and writes share the SMs' way to it (a copy kernel
// with this kernel's loads and stores takes the sum of their times), so an
// expert of up to 256 rows keeps its 128 columns of d in shared memory over a
// run of tiles and streams only x.  The epilogue packs bf16 into swizzled
// shared memory and stores it by TMA, which clips at the weight's own edges.
//
// Qwen2-MoE-shaped gate/up weights (64 x 5120 x 3584, 16384 rows, experts very
// uneven): 729 us for a single call (838 us back to back, at the clock the power
// cap leaves), 2.35 GB written and 0.6 TFLOP; with even experts of at most 256
// rows (12800 rows) 590 us.  The first version, d and x streamed for every tile
// and one 4 KB staging block per warp, took 968 us.  Times in this file are of
// single calls.
//
// Segments are whole multiples of 16 rows (the MMA's K), their padding rows
// zero in both operands; a stage reads up to 63 rows past its segment, but
// only whole 16-row steps inside it are multiplied.  An expert without rows
// gets zeros.  Every wait is bounded as in the other tensor-core kernels.
#include "moe_gemm_host.cuh"

namespace moe {

namespace {

constexpr int kWgThreads = 320;  // TMA warp, MMA warp, 8 epilogue warps
constexpr int kWgEpiWarps = 8;
constexpr int kWgBK = 64;                         // rows per chunk
constexpr int kWgBoxBytes = kWgBK * 128;          // 64 columns x 64 rows
constexpr int kWgOperandBytes = 2 * kWgBoxBytes;  // a CTA's 128 columns of d, or of x, for one chunk
constexpr int kWgPanel = 4;                       // chunks of d held at once
constexpr int kWgRing = 5;                        // chunks of x in flight
constexpr int kWgStoreBytes = 2 * 32 * 128;       // one epilogue warp's 32 x 128 block, as two of 64 columns
constexpr int kWgTableBytes = ((kMaxGroups + 1) * 4 + kMaxGroups * 2 + 255) / 256 * 256;
constexpr int kWgMiscBytes = 256;
constexpr int kWgSmemBytes = 1024 + (kWgPanel + kWgRing) * kWgOperandBytes + kWgEpiWarps * kWgStoreBytes + kWgTableBytes +
                             kWgMiscBytes;
static_assert(kWgSmemBytes <= 227 * 1024, "shared memory");
static_assert((2 * kWgRing + kWgPanel + 5) * 8 + 24 <= kWgMiscBytes, "barriers fit");
static_assert((kWgPanel & (kWgPanel - 1)) == 0, "panel slots by masking");

struct WgradParams {
    const int32_t* seg;
    int n_groups, m, n;
    int d_joined, x_joined;  // tm_d / tm_x load (and tm_out stores) 128 columns in one copy
    int run;                 // tiles along n that an expert of at most 4 chunks takes with one panel of d
    unsigned* status;
    uint64_t wait_limit_ns;
    int withhold_first_load;
};

// One unit of work: `tiles` tiles of 256 x 256 side by side, of one expert.
struct WgItem {
    int g, m0, n0, tiles;
    int row0, steps;   // steps: 16-row MMA steps
};

// The units of one CTA pair, the same sequence for each of its roles.  Experts
// of more than 4 chunks ("streaming", first in `order`) are bound by their
// MMAs and come tile by tile; the others, bound by writing their gradients,
// come in runs of tiles that share a panel of d.  A pair deals itself every
// G-th unit of both lists and mixes them evenly, so that the MMAs of the one
// kind run under the writes of the other.
struct WgSched {
    const int* seg;
    const uint16_t* order;
    int m_tiles, n_tiles, runs, run;
    unsigned n_stream;       // streaming experts
    unsigned s_next, s_left, r_next, r_left, G;
    unsigned acc, total, mine;

    __device__ void init(const WgradParams& p, const int* seg_, const uint16_t* order_, unsigned streaming) {
        seg = seg_;
        order = order_;
        m_tiles = (p.m + 255) / 256;
        n_tiles = (p.n + 255) / 256;
        run = p.run;
        runs = (n_tiles + run - 1) / run;
        n_stream = streaming;
        G = gridDim.x / 2;
        const unsigned pair = blockIdx.x / 2;
        const unsigned ns = streaming * m_tiles * n_tiles, nr = (p.n_groups - streaming) * m_tiles * runs;
        s_next = pair;
        r_next = G - 1 - pair;  // pairs short of one kind get more of the other
        s_left = ns > s_next ? (ns - s_next + G - 1) / G : 0;
        r_left = nr > r_next ? (nr - r_next + G - 1) / G : 0;
        mine = s_left;
        total = s_left + r_left;
        acc = 0;
    }
    __device__ bool next(WgItem& it) {
        if (s_left + r_left == 0) return false;
        acc += mine;
        const bool stream = acc >= total;
        unsigned e, rest;
        if (stream) {
            acc -= total;
            const unsigned per = (unsigned)(m_tiles * n_tiles);
            e = s_next / per;
            rest = s_next - e * per;
            s_next += G;
            --s_left;
            it.tiles = 1;
            const unsigned mt = rest / (unsigned)n_tiles;
            it.m0 = (int)mt * 256;
            it.n0 = (int)(rest - mt * n_tiles) * 256;
        } else {
            const unsigned per = (unsigned)(m_tiles * runs);
            e = r_next / per;
            rest = r_next - e * per;
            e += n_stream;
            r_next += G;
            --r_left;
            const unsigned mt = rest / (unsigned)runs;
            const int first = (int)(rest - mt * runs) * run;
            it.tiles = n_tiles - first < run ? n_tiles - first : run;
            it.m0 = (int)mt * 256;
            it.n0 = first * 256;
        }
        it.g = order[e];
        it.row0 = seg[it.g];
        const int rows = seg[it.g + 1] - it.row0;
        it.steps = rows > 0 ? rows / 16 : 0;
        return true;
    }
};

__global__ void __launch_bounds__(kWgThreads, 1)
    moe_wgrad_kernel(const __grid_constant__ CUtensorMap tm_d, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ CUtensorMap tm_out128,
                     const WgradParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* panel = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = panel + kWgPanel * kWgOperandBytes;
    uint8_t* store_base = ring + kWgRing * kWgOperandBytes;
    int* seg = reinterpret_cast<int*>(store_base + kWgEpiWarps * kWgStoreBytes);
    uint16_t* order = reinterpret_cast<uint16_t*>(seg + kMaxGroups + 1);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(seg) + kWgTableBytes);
    uint64_t* empty = full + kWgRing;     // a chunk of x is free
    uint64_t* pempty = empty + kWgRing;   // a chunk of d is free
    uint64_t* tfull = pempty + kWgPanel;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain_bar = tempty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    unsigned* n_stream = reinterpret_cast<unsigned*>(tmem_holder + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kWgRing; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kWgPanel; ++s) mbar_init(&pempty[s], 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kWgEpiWarps);
        }
        mbar_init(drain_bar, 1);
        fence_barrier_init();
        *abort_flag = 0;
        *n_stream = 0;
        tma_prefetch_desc(&tm_d);
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_out);
        tma_prefetch_desc(&tm_out128);
    }
    if (warp == 1) tmem_alloc_pair(tmem_holder, 512);
    cluster_sync_all();  // the peer's barriers are initialised before any TMA or commit targets them
    pdl_wait();
    for (int g = threadIdx.x; g <= p.n_groups; g += blockDim.x) seg[g] = p.seg[g];
    __syncthreads();
    // experts by descending row count, the lower index first among equals
    for (int g = threadIdx.x; g < p.n_groups; g += blockDim.x) {
        const int rows = seg[g + 1] - seg[g];
        int place = 0;
        for (int o = 0; o < p.n_groups; ++o) {
            const int ro = seg[o + 1] - seg[o];
            place += ro > rows || (ro == rows && o < g);
        }
        order[place] = (uint16_t)g;
        if (rows > kWgPanel * kWgBK) atomicAdd(n_stream, 1u);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    WgSched sch;
    sch.init(p, seg, order, *n_stream);
    WgItem it;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();
            int fills[kWgRing];
#pragma unroll
            for (int s = 0; s < kWgRing; ++s) fills[s] = 0;
            uint32_t s = 0, ph = 0;  // ring cursor
            uint32_t pc = 0;         // panel chunks loaded so far
            bool withhold = p.withhold_first_load && blockIdx.x == 0;
            bool ok = true;
            while (ok && sch.next(it)) {
                const int dc = it.m0 + (int)rank * 128;
                for (int j = 0; ok && j < it.tiles; ++j) {
                    const int xc = it.n0 + j * 256 + (int)rank * 128;
                    const bool load_d = j == 0;  // a streaming unit is one tile
                    for (int k = 0; k < it.steps; k += 4) {
                        if (!mbar_wait_bounded(&empty[s], ph ^ 1u, p.wait_limit_ns, abort_flag) ||
                            (load_d && !mbar_wait_bounded(&pempty[pc % kWgPanel], ((pc / kWgPanel) & 1u) ^ 1u,
                                                          p.wait_limit_ns, abort_flag))) {
                            ok = false;
                            break;
                        }
                        if (withhold) {  // test hook: this chunk is never filled
                            withhold = false;
                        } else {
                            const int row = it.row0 + 16 * k;
                            if (rank == 0)
                                mbar_arrive_expect_tx(&full[s], (load_d ? 4 : 2) * kWgOperandBytes);
                            const uint32_t fb = map_to_rank(smem_u32(&full[s]), 0);
                            // one copy per operand where its rows are whole 64-column blocks: the
                            // issuing thread takes 50-90 ns per copy, a chunk's MMAs 270 ns
                            if (load_d) {
                                uint8_t* dst = panel + (pc % kWgPanel) * kWgOperandBytes;
                                if (p.d_joined) {
                                    tma_load_4d_pair(dst, &tm_d, fb, 0, row, dc / 64, 0, pol);
                                } else {
                                    tma_load_2d_pair(dst, &tm_d, fb, dc, row, pol);
                                    tma_load_2d_pair(dst + kWgBoxBytes, &tm_d, fb, dc + 64, row, pol);
                                }
                            }
                            uint8_t* dst = ring + s * kWgOperandBytes;
                            if (p.x_joined) {
                                tma_load_4d_pair(dst, &tm_x, fb, 0, row, xc / 64, 0, pol);
                            } else {
                                tma_load_2d_pair(dst, &tm_x, fb, xc, row, pol);
                                tma_load_2d_pair(dst + kWgBoxBytes, &tm_x, fb, xc + 64, row, pol);
                            }
                            ++fills[s];
                        }
                        if (load_d) ++pc;
                        if (++s == kWgRing) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
            }
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.status, kStatusTimeout);
            }
            // every issued copy lands before the block exits
            if (rank == 0)
                for (int q = 0; q < kWgRing; ++q)
                    if (fills[q] > 0) mbar_drain(&full[q], (uint32_t)(fills[q] - 1) & 1u, p.wait_limit_ns);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // One thread has 512 cycles to issue a chunk's four MMAs and its
            // commits: descriptors and the cursors are kept incrementally and one
            // commit frees a chunk in both CTAs (recomputing them and committing
            // to each CTA by itself took 705 cycles a chunk; this takes 530).
            uint32_t ac = 0, s = 0, ph = 0, pc = 0;
            bool ok = true;
            const uint32_t idesc = umma_idesc(Elt<__nv_bfloat16>::kMmaFmt, 256, 256) | kIdescAMn | kIdescBMn;
            const uint64_t a_base = umma_desc_mn_sw128<kWgBK>(smem_u32(panel));
            const uint64_t x_base = umma_desc_mn_sw128<kWgBK>(smem_u32(ring));
            constexpr uint32_t kStep = 16 * 128 / 16;  // 16 rows of 128 bytes
            while (ok && sch.next(it)) {
                if (it.steps == 0) continue;
                for (int j = 0; ok && j < it.tiles; ++j) {
                    const int b = ac & 1;
                    if (!mbar_wait_bounded(&tempty[b], ((ac >> 1) & 1u) ^ 1u, p.wait_limit_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t acc = tmem_base + b * 256;
                    const bool last = j + 1 == it.tiles;  // the panel's chunks are free after it
                    uint32_t accumulate = 0, slot = pc;
                    for (int left = it.steps; left > 0; left -= 4, ++slot) {
                        if (!mbar_wait_bounded(&full[s], ph, p.wait_limit_ns, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t a = a_base + (slot % kWgPanel) * (kWgOperandBytes >> 4);
                        const uint64_t x = x_base + s * (kWgOperandBytes >> 4);
                        if (left >= 4) {
                            umma_pair_bf16(acc, a, x, idesc, accumulate);
                            umma_pair_bf16(acc, a + kStep, x + kStep, idesc, 1u);
                            umma_pair_bf16(acc, a + 2 * kStep, x + 2 * kStep, idesc, 1u);
                            umma_pair_bf16(acc, a + 3 * kStep, x + 3 * kStep, idesc, 1u);
                        } else {
                            for (int kk = 0; kk < left; ++kk) {
                                umma_pair_bf16(acc, a + kk * kStep, x + kk * kStep, idesc, accumulate);
                                accumulate = 1;
                            }
                        }
                        accumulate = 1;
                        umma_commit_pair_both(&empty[s]);
                        if (last) umma_commit_pair_both(&pempty[slot % kWgPanel]);
                        if (++s == kWgRing) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                    if (!ok) break;
                    if (last) pc = slot;
                    umma_commit_pair_both(&tfull[b]);
                    ++ac;
                }
            }
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.status, kStatusTimeout);
                umma_commit_pair(smem_u32(drain_bar));
                mbar_drain(drain_bar, 0, p.wait_limit_ns);
            }
        }
    } else {
        const int quad = warp & 3;           // TMEM lanes this warp may access
        const int half = (warp - 2) >> 2;    // 128 of the tile's 256 columns
        uint8_t* mine = store_base + (warp - 2) * kWgStoreBytes;
        const uint64_t pol_out = policy_evict_first();  // written once: the operands keep L2
        uint32_t ac = 0;
        bool ok = true, was_together = false;
        while (ok && sch.next(it)) {
            for (int j = 0; j < it.tiles; ++j) {
                const int b = ac & 1;
                if (it.steps > 0) {
                    // a half's warps meet at barriers below: all go on, or all leave
                    const bool got = mbar_wait_bounded(&tfull[b], (ac >> 1) & 1u, p.wait_limit_ns, abort_flag);
                    if (!named_all(1 + half, 128, got)) {
                        *abort_flag = 1;
                        if (lane == 0) atomicOr(p.status, kStatusTimeout);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                const int row = it.m0 + (int)rank * 128 + quad * 32, col = it.n0 + j * 256 + half * 128;
                // the whole share into registers, packed, and the accumulator freed
                // for the tile after the next
                uint32_t w[64];
                if (it.steps > 0) {
                    const uint32_t ta =
                        tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + b * 256 + half * 128;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld32_nowait(ta + c * 32, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const __nv_bfloat162 h2 =
                                __floats2bfloat162_rn(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                            w[c * 16 + i] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive(&tempty[b]);
                        else mbar_arrive_cluster(map_to_rank(smem_u32(&tempty[b]), 0));
                    }
                    ++ac;
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i) w[i] = 0u;
                }
                // more than 64 rows, columns in whole blocks of 64: the half's four warps
                // store 128 x 128 in one copy (a copy costs the TMA unit 65 ns and 0.7 ns
                // a 128-byte row; with a copy a warp, stores took a third of a tile's time:
                // 12800 rows in 64 experts, 627 us against 590 us).  Few rows are bound by
                // the epilogue's latency: a warp stores its own 32 rows without meeting the
                // others (512 rows in 64 experts: 414 us against 430 us)
                const bool together = p.x_joined && it.steps > 4;
                uint8_t* blk = together ? store_base + half * (4 * kWgStoreBytes) + quad * (32 * 128) : mine;
                const int chunk = together ? 128 * 128 : 32 * 128;  // from one 64-column block to the next
                if (lane == 0) bulk_wait_read();  // this thread's stores have read the staging
                if (together || was_together) named_sync(1 + half, 128);
                else __syncwarp();
                was_together = together;
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    *reinterpret_cast<int4*>(blk + (q >> 3) * chunk + lane * 128 + (((q & 7) ^ (lane & 7)) * 16)) =
                        make_int4((int)w[4 * q], (int)w[4 * q + 1], (int)w[4 * q + 2], (int)w[4 * q + 3]);
                fence_proxy_async_shared();
                if (together) {
                    named_sync(1 + half, 128);
                    if (lane == 0 && quad == 0 && row < p.m && col < p.n) {
                        tma_store_4d(&tm_out128, blk, 0, row, col / 64, it.g, pol_out);
                        bulk_commit();
                    }
                } else {
                    __syncwarp();
                    if (lane == 0 && row < p.m) {
                        if (p.x_joined) {
                            if (col < p.n) tma_store_4d(&tm_out, blk, 0, row, col / 64, it.g, pol_out);
                        } else {
                            if (col < p.n) tma_store_3d(&tm_out, blk, col, row, it.g, pol_out);
                            if (col + 64 < p.n) tma_store_3d(&tm_out, blk + chunk, col + 64, row, it.g, pol_out);
                        }
                        bulk_commit();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    }

    tc_fence_before();
    cluster_sync_all();  // neither CTA frees TMEM or leaves while the pair's MMAs may run
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace

int launch_wgrad(const WgradLaunch& L, const GemmCtl& ctl, cudaStream_t stream) {
    DeviceInfo d;
    int rc = current_device(&d);
    if (rc != 0) return rc;
    if (L.n_groups < 1 || L.n_groups > kMaxGroups || L.m <= 0 || L.n <= 0 || L.rows <= 0) return -1;
    static std::atomic<int> cache[kMaxCachedDevices];
    int blocks = 0;
    if ((rc = resident_blocks(moe_wgrad_kernel, kWgSmemBytes, kWgThreads, 2, d, cache, &blocks)) != 0) return rc;
    CUtensorMap tm_d, tm_x, tm_out, tm_out128;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int dj = L.m % 64 == 0, xj = L.n % 64 == 0;
    if (!(dj ? make_map_cols(&tm_d, dt, L.d, 1, L.rows, L.m, kWgBK, 2) : make_map(&tm_d, dt, 2, L.d, L.rows, L.m, kWgBK)) ||
        !(xj ? make_map_cols(&tm_x, dt, L.x, 1, L.rows, L.n, kWgBK, 2) : make_map(&tm_x, dt, 2, L.x, L.rows, L.n, kWgBK)) ||
        !(xj ? make_map_cols(&tm_out, dt, L.out, L.n_groups, L.m, L.n, 32, 2) &&
                   make_map_cols(&tm_out128, dt, L.out, L.n_groups, L.m, L.n, 128, 2)
             : make_map3(&tm_out, dt, 2, L.out, L.n_groups, L.m, L.n, 32)))
        return -3;
    if (!xj) tm_out128 = tm_out;  // not used
    const long long n_tiles = (L.n + 255) / 256, tiles = (long long)((L.m + 255) / 256) * n_tiles;
    if (tiles * L.n_groups > 0x7fffffffLL - d.num_sms) return -1;
    if (2 * tiles * L.n_groups < blocks) blocks = (int)(2 * tiles * L.n_groups);
    // runs as long as they leave every pair eight units
    long long run = tiles * L.n_groups / (8LL * (blocks / 2));
    run = run < 1 ? 1 : (run > n_tiles ? n_tiles : run);
    WgradParams p{L.seg_offsets, L.n_groups, L.m, L.n, dj, xj, (int)run, ctl.status, wait_limit_ns(),
                  take_withhold_flag()};
    const cudaError_t e = launch_kernel_cluster(moe_wgrad_kernel, dim3(blocks), dim3(kWgThreads), kWgSmemBytes, stream,
                                                2, tm_d, tm_x, tm_out, tm_out128, p);
    count_launch();
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? 0 : -3;
}

}  // namespace moe
