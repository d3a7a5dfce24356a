// CTAs that share a request in the eviction's selection.
#pragma once

namespace smla {

constexpr int kEvictPortableCluster = 8, kEvictMostCluster = 16;
constexpr int kEvictKeySlots = 40960;     // slots of a CTA whose keys fit into shared memory
// A request takes another CTA per so many slots.  (1 x 32768 slots: 4 CTAs 23.5 us, 8 CTAs 30, whole calls.)
constexpr int kEvictSlotsPerCta = 8192;

// `most`: the largest cluster that the device can hold (a GPC may have fewer SMs than 16, and a part of a device fewer still).
inline int evict_cluster(int requests, int cols, int sms, int most) {
  // one CTA per kEvictSlotsPerCta slots, while the requests leave SMs for them
  int csize = 1;
  while (csize < kEvictPortableCluster && csize < most && (long long)requests * csize * 2 <= sms &&
         cols > (long long)csize * kEvictSlotsPerCta)
    csize *= 2;
  // and the largest cluster where the keys do not fit otherwise (1 x 500000 slots: 153 us with 8 CTAs that read them anew for
  // each pass)
  if (csize == kEvictPortableCluster && most >= kEvictMostCluster && (long long)requests * kEvictMostCluster <= sms &&
      cols > (long long)csize * kEvictKeySlots)
    csize = kEvictMostCluster;
  return csize;
}

}  // namespace smla
