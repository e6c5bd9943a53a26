// Which kernels the head's operators take: rules on sizes alone, in plain C++, so that the host can be asked as well
// (tests check by them that they reach each variant).
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace mq {

// ------------------------------------------------------------ the product
// How a product is run: a rule on sizes alone.
struct Linear8Plan {
  int nt;              // blocks of 16 tokens of the kernel that streams the weights; 0: the tiled kernel
  int r;               // its blocks of 16 weight rows a workgroup, or of the tiled kernel a wave
  int waves;           // its waves a workgroup
  int tb;              // blocks of 16 tokens of the tiled kernel
  int splits;          // of the tiled kernel along K
  int per;             // blocks of 128 columns a split, a multiple of 4
  int64_t groups;      // workgroups in all, of 256 threads
  size_t bytes;        // workspace
};

// The tiled kernel's variants, and the time of a step of 128 columns on a CU that has nothing else, in us (MI355X, by 2 to 14
// tiles a CU of 28672 x 8192, two workgroups at a time, which take twice that each).
struct Variant {
  int r, tb;
  double step;
};
constexpr Variant kVariants[] = {{1, 2, 0.165}, {1, 4, 0.29}, {2, 2, 0.27}, {2, 4, 0.36}, {2, 8, 0.54}, {4, 8, 0.97}};

// Up to 16 tokens the weights are streamed. Above, the variant with the least time by a model of what was measured over 17
// to 2048 tokens, 1000 x 1000 to 28672 x 8192 (its choice is the fastest or within a fifth of it): 4 us to begin and end,
// the steps of a CU's tiles one after the other, the weights from memory at 15 TB/s (what is left of it where the steps
// cover the rest), and 5 us and the traffic of partial sums at 5 TB/s to join splits of K. Streamed: 3 us, the weights at
// 5.2 TB/s and the tokens' codes, which each workgroup reads, at 60, by two blocks of weight rows where by one it would be
// more workgroups than CUs (LDS holds one workgroup of 32 tokens: 6144 x 6144 10.4 us by two, 12.7 by one; 4096 x 4096 7.2
// and 6.7), and up to 16 tokens where by two it is four a CU (8 tokens, 65536 x 2048: 24.8 and 25.5; 28672 x 8192: 44.5
// and 42.2). Up to 16 tokens nothing is compared: narrow layers with a long K stay on few CUs (128 x 16384 6.6 us for 2 MB).
inline Linear8Plan plan_linear8(int64_t M, int64_t N, int64_t K) {
  Linear8Plan best = {};
  const int64_t Nb = (N + 15) / 16, Kt = (K + 127) / 128, Kq = (Kt + 3) / 4;
  const double weights = (double)Nb * Kt * 2048;      // bytes of their codes
  double least = 1e30;
  if (M <= 32) {
    best.nt = M <= 16 ? 1 : 2;
    best.r = Nb > (M <= 16 ? 2047 : 256) ? 2 : 1;
    best.waves = (int)(Kq < 8 ? Kq : 8);
    best.groups = 2 * ((Nb + best.r - 1) / best.r);     // of 512 threads
    least = 3.0 + weights / 5.2e6 + (double)Nb / best.r * 16.0 * best.nt * K / 60e6;
    if (M <= 16) return best;
  }
  for (const Variant& v : kVariants) {
    const int64_t T = ((Nb + 4 * v.r - 1) / (4 * v.r)) * ((M + 16 * v.tb - 1) / (16 * v.tb));
    for (int64_t S : {1, 2, 3, 4, 8}) {
      if (S > 1 && (S > Kq || T * S > 1024)) break;
      const int64_t per = (Kq + S - 1) / S, splits = (Kq + per - 1) / per, a_cu = (T * splits + 255) / 256;
      double t = 4.0 + 4.0 * per * a_cu * v.step + weights / 15e6;
      if (splits > 1) t += 5.0 + 8.0 * splits * M * N / 5e6;
      if (t >= least) continue;
      least = t;
      best = {};
      best.r = v.r;
      best.tb = v.tb;
      best.splits = (int)splits;
      best.per = (int)(4 * per);
      best.groups = T * splits;
      if (splits > 1) best.bytes = (size_t)splits * M * N * sizeof(float);
    }
  }
  return best;
}

// ---------------------------------------------------------------- sampling
constexpr int kGroupWaves = 8;             // waves of a workgroup where rows go over the whole GPU, a segment each
constexpr int kMostSegs = 512;             // segments of a row
constexpr int64_t kRowMost = 16384;        // tokens of a row that one workgroup takes,
constexpr int64_t kRowMostEach = 320;      // of several rows this many times the rows,
constexpr int64_t kManyRows = 192, kManyMost = 512 * kMostSegs;      // and of each of many rows

// Segments of a row, of 512 tokens at least: so many that about kGroups workgroups share the rows, and a wave's lanes can
// hold what each workgroup of a row found. (With 256 workgroups 64 x 131072 takes 49 us, so 43.5; 16 x 131072 28.7 and 30.4:
// there the joining of 32 histograms a row takes half of k_weigh.)
constexpr int64_t kGroups = 512;

inline void split(int64_t rows, int64_t vocab, int* splits, int* span) {
  int64_t s = 512;
  auto groups = [&] { return (vocab + kGroupWaves * s - 1) / (kGroupWaves * s); };
  while (groups() > kMostSegs / kGroupWaves || (groups() > 1 && rows * groups() > kGroups)) s *= 2;
  *span = (int)s;
  *splits = (int)groups();
}

// Whether a workgroup takes a row. It takes the same time however many others there are, up to one a CU; over the whole GPU
// rows share it. By rows and over the GPU, in us, top-k 50 with top-p 0.9 and top-p alone: 1 row of 16384 16.1 and 18.2,
// 18.7 and 18.6; of 20000 17.6 and 18.7, 21.7 and 18.4; 64 of 20000 18.8 and 24.1, 22.7 and 25.9; of 32000 23.1 and 26.1,
// 30.3 and 28.8; 128 of 32000 23.2 and 27.3, 30.5 and 32.8; of 50257 31.3 and 30.7, 42.9 and 38.6; 192 of 50257 31.1 and
// 40.1, 43.0 and 56.0.
inline bool by_rows(int64_t rows, int64_t vocab) {
  if (rows >= kManyRows) return vocab <= kManyMost;
  return vocab <= kRowMost || vocab <= kRowMostEach * rows;
}

}  // namespace mq
