// The statements of one output tile, included as the body of gemm_tile_kernel
// and of tile_body (gemm_tile_impl.h), which name the operands and sizes, the
// tile's m0, n0 and K range `split` of kchunk, and the template parameters. Not
// a function that both call: inlined from one, the compiler simplifies the
// loops twice and hoists more addresses out of them. Row-major B then takes 127
// registers instead of 97 in the FP8 64 x 64 kernel (3 waves per SIMD instead of
// 4; 2001 x 2003 x 2005: 219 us against 213) and spills in the 256 x 256 ones.
    using T = Tile<ES, BM, BN, BK, WM, WN, BT>;
    __shared__ __attribute__((aligned(16))) uint8_t smem_raw[2 * T::STAGE];
    LDS_AS uint8_t* smem = (LDS_AS uint8_t*)smem_raw;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;

    const bool interior_mn = aligned && (m0 + BM <= M) && (n0 + BN <= N);
    // Split-K: a workgroup sums K range [kbeg, kend) (the whole of K when the
    // launch is not split). kbeg is a multiple of BK.
    const int kbeg = split * kchunk;
    const int klen = min(K - kbeg, kchunk);
    const int kend = kbeg + klen;

    // This thread's chunk coordinates inside a staged tile.
    const int a_row = tid / T::A_CPR, a_col = tid % T::A_CPR;  // + i * A_RPP rows
    const int b_row = tid / T::B_CPR, b_col = tid % T::B_CPR;  // + i * B_RPP rows

    v4u ra[T::CA];
    v4u rb[T::CB];

    v4f acc[T::TM][T::TN];
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

    const int g = lane >> 4;    // 16-lane group: selects the k sub-range of an operand
    const int j16 = lane & 15;  // lane within its group
    // B transpose-read pattern (lane maps measured for ds_read_b64_tr_b16 /
    // _b8: lane i of a 16-lane group receives element i % E of lanes
    // (16/E)*e + i/E, E = elements per 64 bits).
    const int b_row_in = (ES == 2) ? (j16 >> 2) : (j16 >> 1);
    const int b_col_in = (ES == 2) ? 4 * (j16 & 3) : 8 * (j16 & 1);
    // Operand reads: row of this lane (+ stage + tm*16*SA) and byte offset in
    // the row (g*OPB + ks*KPI*ES, through rd below).
    const int a_lds = (wm * T::WTM + j16) * T::SA;
    const int goff = g * T::OPB;
    // BT: row of this lane + stage + tn*16*SA, offsets as for A
    const int b_lds = BT ? (wn * T::WTN + j16) * T::SA
                         : T::b_row(8 * (ES == 2 ? 1 : 4) * g + b_row_in)  // + stage + b_row(ks*KPI) + tn*16*ES
                               + (wn * T::WTN + b_col_in) * ES;

    const int nk = (klen + BK - 1) / BK;
    typedef typename Operand<ES>::type Op;

    // ---- global <-> registers <-> LDS (A and B have separate stages) ----
    // Fast-path loads: a wave-uniform base (kept in SGPRs) plus a 32-bit
    // per-lane offset, so the 16 loads of a tile need no 64-bit VGPR addresses.
    // Valid while one tile row block spans less than 2^31 bytes (checked below).
    const uint8_t* a_tile = A + ((int64_t)m0 * K + kbeg) * GES;
    const uint8_t* b_tile = BT ? B + ((int64_t)n0 * K + kbeg) * GES : B + ((int64_t)kbeg * N + n0) * GES;
    constexpr bool kWiden = GES != ES;
    const bool a_e5m2 = (eflags & EPI_A_E5M2) != 0, b_e5m2 = (eflags & EPI_B_E5M2) != 0;
    // One staged 16-byte chunk from global memory at p (VE elements).
    auto gload = [&](const uint8_t* p, bool e5m2) __attribute__((always_inline)) -> v4u {
        if constexpr (kWiden) {
            const v2i w = *reinterpret_cast<const v2i*>(p);
            return widen8_fp8((uint32_t)w.x, (uint32_t)w.y, e5m2);
        } else if constexpr (UA) {
            return *reinterpret_cast<const v4u_any*>(p);
        } else {
            return *reinterpret_cast<const v4u*>(p);
        }
    };
    auto gload_guarded = [&](const uint8_t* row_ptr, bool row_ok, int64_t col, int64_t limit, bool e5m2)
        __attribute__((always_inline)) -> v4u {
        if constexpr (kWiden) {
            const v2i w = load_codes8_guarded(row_ptr, row_ok, col, limit);
            return widen8_fp8((uint32_t)w.x, (uint32_t)w.y, e5m2);
        } else if constexpr (UA) {
            return load_chunk_any<ES>(row_ptr, row_ok, col, limit);
        } else {
            return load_chunk_guarded<ES>(row_ptr, row_ok, col, limit);
        }
    };
    // Edge tiles (aligned operands) use the same unguarded loads with the
    // addresses clamped into the matrix: A rows past M re-read row M-1 and B
    // column chunks past N re-read the last chunk. Those values only reach
    // output rows/columns that are never stored, and every address is valid.
    uint32_t a_offs[T::CA], b_offs[T::CB];
#pragma unroll
    for (int i = 0; i < T::CA; ++i) {
        const int r = min(m0 + a_row + i * T::A_RPP, M - 1) - m0;
        a_offs[i] = (uint32_t)((r * K + a_col * T::VE) * GES);
    }
#pragma unroll
    for (int i = 0; i < T::CB; ++i) {
        if constexpr (BT) {
            const int r = min(n0 + b_row + i * T::B_RPP, N - 1) - n0;
            b_offs[i] = (uint32_t)((r * K + b_col * T::VE) * GES);
        } else {
            const int c = (UA ? max(min(n0 + b_col * T::VE, N - T::VE), 0) : min(n0 + b_col * T::VE, N - T::VE)) - n0;
            b_offs[i] = (uint32_t)(((b_row + i * T::B_RPP) * N + c) * GES);
        }
    }
    auto load_a = [&](int kt) __attribute__((always_inline)) {
        const uint8_t* pa = a_tile + (int64_t)kt * BK * GES;
#pragma unroll
        for (int i = 0; i < T::CA; ++i) ra[i] = gload(pa + a_offs[i], a_e5m2);
    };
    auto load_b = [&](int kt) __attribute__((always_inline)) {
        const uint8_t* pb = b_tile + (BT ? (int64_t)kt * BK * GES : (int64_t)kt * BK * N * GES);
#pragma unroll
        for (int i = 0; i < T::CB; ++i) rb[i] = gload(pb + b_offs[i], b_e5m2);
    };
    auto store_a = [&](int stage) __attribute__((always_inline)) {
        LDS_AS uint8_t* As = smem + T::a_stage(stage);
#pragma unroll
        for (int i = 0; i < T::CA; ++i)
            *(LDS_AS v4u*)(As + (a_row + i * T::A_RPP) * T::SA + T::chunk(a_row, a_col)) = ra[i];
    };
    auto store_b = [&](int stage) __attribute__((always_inline)) {
        LDS_AS uint8_t* Bs = smem + T::b_stage(stage);
#pragma unroll
        for (int i = 0; i < T::CB; ++i)
            *(LDS_AS v4u*)(Bs + T::b_row(b_row + i * T::B_RPP) + T::chunk(b_row, b_col)) = rb[i];
    };
    // Edge tiles, the K tail and unaligned operands: each 16-byte chunk is
    // loaded with per-element guards and written straight to LDS (no register
    // staging, and a rolled loop, so this path costs almost no registers).
    auto guarded_to_lds = [&](int kt, int stage) __attribute__((always_inline)) {
        const int k0 = kbeg + kt * BK;
        LDS_AS uint8_t* As = smem + T::a_stage(stage);
        LDS_AS uint8_t* Bs = smem + T::b_stage(stage);
#pragma unroll 1
        for (int i = 0; i < T::CA; ++i) {
            const int gm = m0 + a_row + i * T::A_RPP;
            const int64_t gk = (int64_t)k0 + a_col * T::VE;
            const uint8_t* rp = A + (int64_t)gm * K * GES;
            v4u v;
            if (aligned && gm < M && gk + T::VE <= kend)
                v = gload(rp + gk * GES, a_e5m2);
            else
                v = gload_guarded(rp, gm < M, gk, kend, a_e5m2);
            *(LDS_AS v4u*)(As + (a_row + i * T::A_RPP) * T::SA + T::chunk(a_row, a_col)) = v;
        }
#pragma unroll 1
        for (int i = 0; i < T::CB; ++i) {
            if constexpr (BT) {
                const int gn = n0 + b_row + i * T::B_RPP;
                const int64_t gk = (int64_t)k0 + b_col * T::VE;
                const uint8_t* rp = B + (int64_t)gn * K * GES;
                v4u v;
                if (aligned && gn < N && gk + T::VE <= kend)
                    v = gload(rp + gk * GES, b_e5m2);
                else
                    v = gload_guarded(rp, gn < N, gk, kend, b_e5m2);
                *(LDS_AS v4u*)(Bs + T::b_row(b_row + i * T::B_RPP) + T::chunk(b_row, b_col)) = v;
                continue;
            }
            const int gk = k0 + b_row + i * T::B_RPP;
            const int64_t gn = (int64_t)n0 + b_col * T::VE;
            const uint8_t* rp = B + (int64_t)gk * N * GES;
            v4u v;
            if (aligned && gk < kend && gn + T::VE <= N)
                v = gload(rp + gn * GES, b_e5m2);
            else
                v = gload_guarded(rp, gk < kend, gn, N, b_e5m2);
            *(LDS_AS v4u*)(Bs + T::b_row(b_row + i * T::B_RPP) + T::chunk(b_row, b_col)) = v;
        }
    };

    // ---- LDS -> MFMA operands ----
    // One operand (OPB bytes) at byte offset off of an LDS row; rows of a row
    // block start at multiples of 16, so the swizzle of this lane's row is j16/2.
    const int rsw = j16 >> 1;
    auto rd = [&](const LDS_AS uint8_t* rowp, int off) __attribute__((always_inline)) -> Op {
        if constexpr (T::SWZ) {
            const int q = off >> 4;
            if constexpr (ES == 1) {
                // The 32 codes of k-group g are chunks g and g + 4 of the row
                // (A and B alike, so the sum over k is unchanged; every aligned
                // group of 8 k the FP8 matrix cores add together is still 8
                // consecutive k). Two adjacent chunks per lane left about 3
                // bank-conflict cycles per LDS read; this split leaves none.
                const int q0 = q >> 1;
                const v4i lo = *(const LDS_AS v4i*)(rowp + ((q0 ^ rsw) << 4));
                const v4i hi = *(const LDS_AS v4i*)(rowp + (((q0 + 4) ^ rsw) << 4));
                return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
                return __builtin_bit_cast(v8h, *(const LDS_AS v4u*)(rowp + ((q ^ rsw) << 4)));
            }
        } else {
            return Operand<ES>::read_a(rowp + off);
        }
    };
    auto read_b = [&](int stage, Op (&bop)[T::KS][T::TN]) __attribute__((always_inline)) {
        const LDS_AS uint8_t* base = smem + T::b_stage(stage) + b_lds;
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks)
#pragma unroll
            for (int tn = 0; tn < T::TN; ++tn) {
                if constexpr (BT)
                    bop[ks][tn] = rd(base + tn * 16 * T::SA, goff + ks * T::KPI * ES);
                else
                    bop[ks][tn] = Operand<ES>::read_b(base + T::b_row(ks * T::KPI) + tn * 16 * ES, T::SB);
            }
    };
    auto mma_tile = [&](int stage, const Op (&bop)[T::KS][T::TN]) __attribute__((always_inline)) {
        const LDS_AS uint8_t* base = smem + T::a_stage(stage) + a_lds;
        if constexpr (kPrefetchA<BT> && T::NT > 256) {
            // Row blocks in (ks, tm) order; the A operand of the next block is
            // read before this block's MFMAs, so its LDS latency runs under them.
            constexpr int NB = T::KS * T::TM;
            auto a_read = [&](int b) { return rd(base + (b % T::TM) * 16 * T::SA, goff + (b / T::TM) * T::KPI * ES); };
            Op acur = a_read(0);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int ks = b / T::TM, tm = b % T::TM;
                const Op anext = a_read(b + 1 < NB ? b + 1 : b);
                if constexpr (kMfmaPrio<BT>) __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int tn = 0; tn < T::TN; ++tn)
                    acc[tm][tn] = Operand<ES>::template mma<FA, FB>(acur, bop[ks][tn], acc[tm][tn]);
                if constexpr (kMfmaPrio<BT>) __builtin_amdgcn_s_setprio(0);
#pragma unroll
                for (int tn = 0; tn < T::TN; ++tn) asm volatile("" : "+v"(acc[tm][tn])::"memory");
                acur = anext;
            }
            return;
        }
#pragma unroll
        for (int ks = 0; ks < T::KS; ++ks)
#pragma unroll
            for (int tm = 0; tm < T::TM; ++tm) {
                const Op aop = rd(base + tm * 16 * T::SA, goff + ks * T::KPI * ES);
                if constexpr (kMfmaPrio<BT> && T::NT > 256) __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int tn = 0; tn < T::TN; ++tn) acc[tm][tn] = Operand<ES>::template mma<FA, FB>(aop, bop[ks][tn], acc[tm][tn]);
                if constexpr (kMfmaPrio<BT> && T::NT > 256) __builtin_amdgcn_s_setprio(0);
                // With two waves per SIMD the other wave hides the A read
                // latency. Pinning this row block's products here (an empty
                // asm that reads and rewrites its accumulators, after which no
                // LDS read may be hoisted) keeps one A operand live at a time
                // instead of letting the compiler sink every MFMA to the loop
                // end and hold all A operands.
                if constexpr (T::NT > 256) {
#pragma unroll
                    for (int tn = 0; tn < T::TN; ++tn) asm volatile("" : "+v"(acc[tm][tn])::"memory");
                }
            }
    };

    const bool offsets_fit = (int64_t)BM * K * GES < (1ll << 31) &&
                             (BT ? (int64_t)BN * K * GES : (int64_t)BK * N * GES) < (1ll << 31);
    if constexpr (UA) {
        // D tiles in registers ahead of the LDS, so that a tile has D times the
        // work of one to arrive in. Every load goes out without a condition (a
        // branch around one would make the compiler wait for all of them): past
        // K and N addresses are clamped into the matrix, and what they bring is
        // put right on the way to the LDS. There, chunks of A (and of Bt) that K
        // cuts, the 16 bytes before its end, are shifted down, those past it are
        // zeros, as are rows of a row-major B past K (its last row); column
        // chunks of it that N cuts are shifted too. Only operands narrower than
        // a chunk take the element-wise path.
        constexpr int D = BM <= 64 ? kAhead64 : kAhead128, U = D < 2 ? 2 : D;   // U: tiles unrolled
        const bool wide = offsets_fit && K >= T::VE && (BT || N >= T::VE);
        const int nk_full = klen / BK;
        const bool cut = !BT && n0 + BN > N && N % T::VE != 0;
        auto shifted = [](v4u v, int elements) __attribute__((always_inline)) -> v4u {
            if (elements >= T::VE) return v4u{0u, 0u, 0u, 0u};
            return __builtin_bit_cast(v4u, __builtin_bit_cast(unsigned __int128, v) >> (8 * GES * elements));
        };
        const uint8_t* a_base = A + (int64_t)m0 * K * GES;
        const uint8_t* b_base = BT ? B + (int64_t)n0 * K * GES : B;
        uint32_t a_row_at[T::CA], b_row_at[T::CB];   // bytes to this thread's rows (row-major B: unused)
#pragma unroll
        for (int i = 0; i < T::CA; ++i) a_row_at[i] = (uint32_t)(min(a_row + i * T::A_RPP, M - 1 - m0) * K * GES);
#pragma unroll
        for (int i = 0; i < T::CB; ++i) b_row_at[i] = BT ? (uint32_t)(min(b_row + i * T::B_RPP, N - 1 - n0) * K * GES) : 0u;
        const int b_col_at = BT ? 0 : max(min(n0 + b_col * T::VE, N - T::VE), 0);
        v4u qa[D][T::CA], qb[D][T::CB];
        auto fetch = [&](int kt, int set) __attribute__((always_inline)) {
            const int k0 = min(kt, nk - 1) * BK;   // past the last tile: that one again, unused
            const uint32_t ca = (uint32_t)(min(k0 + a_col * T::VE, K - T::VE) * GES);
#pragma unroll
            for (int i = 0; i < T::CA; ++i) qa[set][i] = gload(a_base + (a_row_at[i] + ca), a_e5m2);
            if constexpr (BT) {
                const uint32_t cb = (uint32_t)(min(k0 + b_col * T::VE, K - T::VE) * GES);
#pragma unroll
                for (int i = 0; i < T::CB; ++i) qb[set][i] = gload(b_base + (b_row_at[i] + cb), b_e5m2);
            } else {
                const uint8_t* pb = b_base + (int64_t)k0 * N * GES;
                const int last = K - 1 - k0;
#pragma unroll
                for (int i = 0; i < T::CB; ++i)
                    qb[set][i] = gload(pb + (uint32_t)((min(b_row + i * T::B_RPP, last) * N + b_col_at) * GES), b_e5m2);
            }
        };
        auto put = [&](int kt, int stage, int set) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < T::CA; ++i) ra[i] = qa[set][i];
#pragma unroll
            for (int i = 0; i < T::CB; ++i) rb[i] = qb[set][i];
            if (kt >= nk_full) {
                const int a_past = max(0, kt * BK + a_col * T::VE + T::VE - K);
                const int b_past = max(0, kt * BK + b_col * T::VE + T::VE - K);
#pragma unroll
                for (int i = 0; i < T::CA; ++i) ra[i] = shifted(ra[i], a_past);
#pragma unroll
                for (int i = 0; i < T::CB; ++i) {
                    if (BT) rb[i] = shifted(rb[i], b_past);
                    else if (kt * BK + b_row + i * T::B_RPP >= K) rb[i] = v4u{0u, 0u, 0u, 0u};
                }
            }
            if (cut) {
                const int past = max(0, n0 + b_col * T::VE + T::VE - N);
#pragma unroll
                for (int i = 0; i < T::CB; ++i) rb[i] = shifted(rb[i], past);
            }
            store_a(stage);
            store_b(stage);
        };
        Op bop[T::KS][T::TN];
        if (!wide) {
#pragma unroll 1
            for (int kt = 0; kt < nk; ++kt) {
                guarded_to_lds(kt, 0);
                __syncthreads();
                read_b(0, bop);
                mma_tile(0, bop);
                __syncthreads();
            }
        } else if (nk > 0) {
#pragma unroll
            for (int u = 0; u < D; ++u) fetch(u, u);
            put(0, 0, 0);
            fetch(D, 0);
            __syncthreads();
            for (int k0 = 0; k0 < nk; k0 += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) {   // tile k0 + u, in LDS stage u % 2
                    if (k0 + u >= nk) break;
                    read_b(u & 1, bop);
                    mma_tile(u & 1, bop);
                    if (k0 + u + 1 < nk) {
                        put(k0 + u + 1, (u + 1) & 1, (u + 1) % D);
                        fetch(k0 + u + 1 + D, (u + 1) % D);
                    }
                    __syncthreads();   // (after the last tile too: the caller may start another on the same LDS)
                }
            }
        }
    } else if (nk > 0) {
        Op bop[T::KS][T::TN];
        // Tile kt+1 is fetched into registers while tile kt is multiplied;
        // the K tail and unaligned operands load each chunk with element
        // guards straight into LDS.
        auto fast = [&](int kt) __attribute__((always_inline)) {
            return aligned && offsets_fit && (kt + 1) * BK <= klen;
        };
        if (fast(0)) {
            load_a(0);
            load_b(0);
            store_a(0);
            store_b(0);
        } else {
            guarded_to_lds(0, 0);
        }
        __syncthreads();
        for (int kt = 0; kt < nk; ++kt) {
            const bool more = kt + 1 < nk;
            const bool fast_next = more && fast(kt + 1);
            if (fast_next) {
                load_a(kt + 1);
                load_b(kt + 1);
            }
            read_b(kt & 1, bop);
            mma_tile(kt & 1, bop);
            if (fast_next) {
                store_a((kt + 1) & 1);
                store_b((kt + 1) & 1);
            } else if (more) {
                guarded_to_lds(kt + 1, (kt + 1) & 1);
            }
            __syncthreads();
        }
    }

    // Epilogue: y = acc * (sA*sB), converted, stored with M/N predication on edge tiles.
    // Per-tensor: y = acc * sA*sB (/ sOut). Per-channel (EPI_CHANNEL, sA[M] and
    // sB[N]): y = acc * (1/sOut) * sA[row] * sB[col], loaded only for stored
    // elements.
    // A split-K partial (EPI_PARTIAL, OUT_F32) stores the raw sum into the
    // split's [M, N] slice of the workspace C.
    const bool partial = (eflags & EPI_PARTIAL) != 0;
    if (partial) C = reinterpret_cast<float*>(C) + (int64_t)split * M * N;
    const bool chan = !partial && (eflags & EPI_CHANNEL) != 0;
    const float scale = partial ? 1.0f : epilogue_base(sA, sB, sOut, OUT == OUT_E4M3, chan);  // both FP8 outputs
    const int row0 = m0 + wm * T::WTM + 4 * g;
    const int col0 = n0 + wn * T::WTN + j16;
    if constexpr (Ext::kActive) {
        // scaled here, added to, stored as it is
#pragma unroll
        for (int tm = 0; tm < T::TM; ++tm)
#pragma unroll
            for (int tn = 0; tn < T::TN; ++tn)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc[tm][tn][r] *= scale;
                    if (chan) acc[tm][tn][r] *= sA[min(row0 + tm * 16 + r, M - 1)] * sB[min(col0 + tn * 16, N - 1)];
                }
        ext.template add16<T::TM, T::TN>(acc, m0 + wm * T::WTM, n0 + wn * T::WTN, M, N);
#pragma unroll
        for (int tm = 0; tm < T::TM; ++tm)
#pragma unroll
            for (int tn = 0; tn < T::TN; ++tn)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = row0 + tm * 16 + r, col = col0 + tn * 16;
                    if (row < M && col < N) store_one<OUT>(C, (int64_t)row * N + col, acc[tm][tn][r], eflags);
                }
        static_assert(BT && GES == ES, "adapters stand beside K-major weights");
        auto product = [&](int row, int col) __attribute__((always_inline)) -> float {
            const uint8_t* pa = A + (int64_t)row * K * ES;
            const uint8_t* pb = B + (int64_t)col * K * ES;
            float sum = 0.0f;
#pragma unroll 1
            for (int k = 0; k < K; ++k) sum = __builtin_fmaf(element<ES, FA>(pa, k), element<ES, FB>(pb, k), sum);
            sum *= scale;
            return chan ? sum * (sA[row] * sB[col]) : sum;
        };
        ext.template repair16<T::TM, T::TN>(
            acc, m0 + wm * T::WTM, n0 + wn * T::WTN, M, N, product,
            [&](int row, int col, float y) { store_one<OUT>(C, (int64_t)row * N + col, y, eflags); });
        return;
    }
    if (interior_mn) {
#pragma unroll
        for (int tm = 0; tm < T::TM; ++tm)
#pragma unroll
            for (int tn = 0; tn < T::TN; ++tn)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = row0 + tm * 16 + r, col = col0 + tn * 16;
                    float y = acc[tm][tn][r] * scale;
                    if (chan) y *= sA[row] * sB[col];
                    store_one<OUT>(C, (int64_t)row * N + col, y, eflags);
                }
    } else {
#pragma unroll
        for (int tm = 0; tm < T::TM; ++tm)
#pragma unroll
            for (int tn = 0; tn < T::TN; ++tn)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = row0 + tm * 16 + r, col = col0 + tn * 16;
                    if (row < M && col < N) {
                        float y = acc[tm][tn][r] * scale;
                        if (chan) y *= sA[row] * sB[col];
                        store_one<OUT>(C, (int64_t)row * N + col, y, eflags);
                    }
                }
    }
