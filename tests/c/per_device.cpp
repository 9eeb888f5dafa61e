// Numbers kept per device: looked up once for each device and index, never taken from another.
#include <cstdio>

#include "launch.h"

int main() {
  static qmoe::PerDevice<3> numbers;
  int asked = 0, bad = 0;
  auto get = [&](int dev, int i, int value) {
    return numbers.get(dev, i, [&] {
      ++asked;
      return value;
    });
  };
  for (int round = 0; round < 2; ++round)
    for (int dev = 0; dev < 3; ++dev)
      for (int i = 0; i < 3; ++i) bad += get(dev, i, 100 * dev + i + 1) != 100 * dev + i + 1;
  bad += asked != 9;
  bad += get(5, 0, -1) != 0;  // a look that fails is not kept
  bad += get(5, 0, 7) != 7;
  bad += get(-1, 0, 7) != 0 || get(qmoe::kMaxDevices, 0, 7) != 0;
  std::printf("%d failure(s)\n", bad);
  return bad != 0;
}
