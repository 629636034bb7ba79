// moe_wgrad.cu -- weight gradients of the experts' products on the sm_100a
// tensor cores: for every expert e, over the rows p of its segment,
//   out[e] [m, n] = sum_p d[p, m] x[p, n]
// (dW2 with d the gradient of the down projection's output and x the
// activations; dW13 with d the gradients of the pre-activations and x the
// permuted tokens).  The reduction runs over the rows, so both operands are
// taken MN-major, as they lie in memory: a TMA box is 64 columns by 64 rows.
//
// A CTA pair computes a 256 x 256 tile with the 2-SM MMA (each CTA stages its
// 128 columns of d and half of the 256 columns of x: 32 KB a stage for 512
// cycles of MMA), two accumulators in TMEM so that the epilogue of one tile
// runs under the MMAs of the next: with a few hundred rows per expert a tile
// has only a handful of k-steps and its 128 KB of output weighs as much as its
// operands.  The epilogue packs bf16 into a swizzled shared-memory tile and
// stores it by TMA, which clips at the weight's own edges.
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
constexpr int kWgBK = 64;                      // rows per stage
constexpr int kWgBoxBytes = kWgBK * 128;       // 64 columns x 64 rows
constexpr int kWgStageBytes = 4 * kWgBoxBytes;  // 128 columns of d, 128 of x
constexpr int kWgStoreBytes = 32 * 128;        // one epilogue warp's 32 x 64 block
constexpr int kWgTableBytes = ((kMaxGroups + 1) * 4 + 255) / 256 * 256;
constexpr int kWgMiscBytes = 256;
constexpr int kWgStages = (227 * 1024 - 1024 - kWgEpiWarps * kWgStoreBytes - kWgTableBytes - kWgMiscBytes) / kWgStageBytes;
constexpr int kWgSmemBytes =
    1024 + kWgStages * kWgStageBytes + kWgEpiWarps * kWgStoreBytes + kWgTableBytes + kWgMiscBytes;
static_assert(kWgStages >= 3 && kWgSmemBytes <= 227 * 1024, "shared memory");
static_assert((2 * kWgStages + 5) * 8 + 16 <= kWgMiscBytes, "barriers fit");

struct WgradParams {
    const int32_t* seg;
    int n_groups, m, n;
    unsigned* status;
    uint64_t wait_limit_ns;
    int withhold_first_load;
};

__global__ void __launch_bounds__(kWgThreads, 1)
    moe_wgrad_kernel(const __grid_constant__ CUtensorMap tm_d, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_out, const WgradParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* store_base = smem + kWgStages * kWgStageBytes;
    int* seg = reinterpret_cast<int*>(store_base + kWgEpiWarps * kWgStoreBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(seg) + kWgTableBytes);
    uint64_t* empty = full + kWgStages;
    uint64_t* tfull = empty + kWgStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain_bar = tempty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kWgStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kWgEpiWarps);
        }
        mbar_init(drain_bar, 1);
        fence_barrier_init();
        *abort_flag = 0;
        tma_prefetch_desc(&tm_d);
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_out);
    }
    if (warp == 1) tmem_alloc_pair(tmem_holder, 512);
    cluster_sync_all();  // the peer's barriers are initialised before any TMA or commit targets them
    pdl_wait();
    for (int g = threadIdx.x; g <= p.n_groups; g += blockDim.x) seg[g] = p.seg[g];
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;

    const int MT = (p.m + 255) / 256, NT = (p.n + 255) / 256;
    const long long total = (long long)p.n_groups * MT * NT;
    const int G = gridDim.x / 2;
    struct Tile {
        int g, m0, n0, row0, steps;  // steps: 16-row MMA steps
    };
    auto tile = [&](long long i) {
        Tile t;
        t.g = (int)(i / ((long long)MT * NT));
        const int r = (int)(i - (long long)t.g * MT * NT);
        t.m0 = r / NT * 256;
        t.n0 = r % NT * 256;
        t.row0 = seg[t.g];
        const int rows = seg[t.g + 1] - t.row0;
        t.steps = rows > 0 ? rows / 16 : 0;
        return t;
    };
    const long long first = blockIdx.x / 2;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();
            int fills[kWgStages];
#pragma unroll
            for (int s = 0; s < kWgStages; ++s) fills[s] = 0;
            uint32_t kc = 0;
            bool withhold = p.withhold_first_load && blockIdx.x == 0;
            bool ok = true;
            for (long long i = first; ok && i < total; i += G) {
                const Tile t = tile(i);
                const int dc = t.m0 + (int)rank * 128, xc = t.n0 + (int)rank * 128;
                for (int k = 0; k < t.steps; k += 4, ++kc) {
                    const int s = kc % kWgStages;
                    const uint32_t ph = (kc / kWgStages) & 1u;
                    if (!mbar_wait_bounded(&empty[s], ph ^ 1u, p.wait_limit_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (withhold) {  // test hook: this stage is never filled
                        withhold = false;
                        continue;
                    }
                    uint8_t* st = smem + s * kWgStageBytes;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kWgStageBytes);
                    const uint32_t fb = map_to_rank(smem_u32(&full[s]), 0);
                    const int row = t.row0 + 16 * k;
                    tma_load_2d_pair(st, &tm_d, fb, dc, row, pol);
                    tma_load_2d_pair(st + kWgBoxBytes, &tm_d, fb, dc + 64, row, pol);
                    tma_load_2d_pair(st + 2 * kWgBoxBytes, &tm_x, fb, xc, row, pol);
                    tma_load_2d_pair(st + 3 * kWgBoxBytes, &tm_x, fb, xc + 64, row, pol);
                    ++fills[s];
                }
            }
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.status, kStatusTimeout);
            }
            // every issued copy lands before the block exits
            if (rank == 0)
                for (int s = 0; s < kWgStages; ++s)
                    if (fills[s] > 0) mbar_drain(&full[s], (uint32_t)(fills[s] - 1) & 1u, p.wait_limit_ns);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            uint32_t kc = 0, ac = 0;
            bool ok = true;
            const uint32_t idesc = umma_idesc(Elt<__nv_bfloat16>::kMmaFmt, 256, 256) | kIdescAMn | kIdescBMn;
            for (long long i = first; ok && i < total; i += G) {
                const Tile t = tile(i);
                if (t.steps == 0) continue;
                const int b = ac & 1;
                if (!mbar_wait_bounded(&tempty[b], ((ac >> 1) & 1u) ^ 1u, p.wait_limit_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem_base + b * 256;
                for (int k = 0; k < t.steps; k += 4, ++kc) {
                    const int s = kc % kWgStages;
                    if (!mbar_wait_bounded(&full[s], (kc / kWgStages) & 1u, p.wait_limit_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = smem_u32(smem + s * kWgStageBytes);
                    const uint64_t a = umma_desc_mn_sw128<kWgBK>(st);
                    const uint64_t x = umma_desc_mn_sw128<kWgBK>(st + 2 * kWgBoxBytes);
                    const int n = t.steps - k < 4 ? t.steps - k : 4;
                    for (int kk = 0; kk < n; ++kk)  // 16 rows of 128 bytes per step
                        umma_pair_bf16(acc, a + kk * (16 * 128 / 16), x + kk * (16 * 128 / 16), idesc,
                                       (k > 0 || kk > 0) ? 1u : 0u);
                    umma_commit_pair(smem_u32(&empty[s]));  // the stage is free in both CTAs
                    umma_commit_pair(map_to_rank(smem_u32(&empty[s]), 1));
                }
                if (!ok) break;
                umma_commit_pair(smem_u32(&tfull[b]));
                umma_commit_pair(map_to_rank(smem_u32(&tfull[b]), 1));
                ++ac;
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
        uint32_t ac = 0;
        for (long long i = first; i < total; i += G) {
            const Tile t = tile(i);
            const int b = ac & 1;
            if (t.steps > 0) {
                const bool got = mbar_wait_bounded(&tfull[b], (ac >> 1) & 1u, p.wait_limit_ns, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    *abort_flag = 1;
                    if (lane == 0) atomicOr(p.status, kStatusTimeout);
                    break;
                }
                tc_fence_after();
            }
            const int row = t.m0 + (int)rank * 128 + quad * 32;
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // 64 columns at a time
                const int col = half * 128 + c * 64;
                uint32_t v[2][32];
                if (t.steps > 0) {
                    const uint32_t ta = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + b * 256 + col;
                    tmem_ld32_nowait(ta, v[0]);
                    tmem_ld32_nowait(ta + 32, v[1]);
                    tmem_wait_ld();
                    if (c == 1) {  // the accumulator is free for the tile after the next
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (rank == 0) mbar_arrive(&tempty[b]);
                            else mbar_arrive_cluster(map_to_rank(smem_u32(&tempty[b]), 0));
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[0][j] = v[1][j] = 0u;
                }
                if (lane == 0) bulk_wait_read();  // the previous store has read this warp's block
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[q >> 2][(q & 3) * 8 + j]);
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t*>(&h2);
                    }
                    *reinterpret_cast<int4*>(mine + lane * 128 + ((q ^ (lane & 7)) * 16)) =
                        make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0 && row < p.m && t.n0 + col < p.n) tma_store_3d(&tm_out, mine, t.n0 + col, row, t.g);
                if (lane == 0) bulk_commit();
            }
            if (t.steps > 0) ++ac;
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
    CUtensorMap tm_d, tm_x, tm_out;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (!make_map(&tm_d, dt, 2, L.d, L.rows, L.m, kWgBK) || !make_map(&tm_x, dt, 2, L.x, L.rows, L.n, kWgBK) ||
        !make_map3(&tm_out, dt, 2, L.out, L.n_groups, L.m, L.n, 32))
        return -3;
    WgradParams p{L.seg_offsets, L.n_groups, L.m, L.n, ctl.status, wait_limit_ns(), take_withhold_flag()};
    const long long tiles = (long long)L.n_groups * ((L.m + 255) / 256) * ((L.n + 255) / 256);
    if (2 * tiles < blocks) blocks = (int)(2 * tiles);
    const cudaError_t e = launch_kernel_cluster(moe_wgrad_kernel, dim3(blocks), dim3(kWgThreads), kWgSmemBytes, stream,
                                                2, tm_d, tm_x, tm_out, p);
    count_launch();
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? 0 : -3;
}

}  // namespace moe
