// Where the keys of selected pages lie (fa_decode.cuh), on the host: "page_size max_pages at sel[0] sel[1] ..." a line in, with the
// entries that may be read, which end where the memory does; the key's position out.
#include <sys/mman.h>
#include <unistd.h>

#include <cstdio>
#include <cstring>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "../flash_attention_backward_gb300/csrc/fa_decode.cuh"

int main() {
  const size_t page = sysconf(_SC_PAGESIZE);
  char* two = static_cast<char*>(mmap(nullptr, 2 * page, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0));
  if (two == MAP_FAILED || mprotect(two + page, page, PROT_NONE) != 0) return 2;
  for (std::string line; std::getline(std::cin, line);) {
    std::istringstream in(line);
    int at;
    fap::Cache c{};
    in >> c.page_size >> c.max_pages >> at;
    fap::page_divisor(c.page_size, &c.page_mul, &c.page_shift);
    std::vector<int32_t> sel;
    for (long long x; in >> x;) sel.push_back((int32_t)x);
    const size_t bytes = sel.size() * sizeof(int32_t);
    if (bytes > page) return 2;
    int32_t* list = reinterpret_cast<int32_t*>(two + page - bytes);
    std::memcpy(list, sel.data(), bytes);
    std::printf("%d\n", fap::selected_position(c, list, (int)sel.size() * c.page_size, at));
  }
}
